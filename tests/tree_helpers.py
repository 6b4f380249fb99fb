"""Trees of drafted tokens for the tests: ancestors, masks and expected results
by plain walks, attention by the oracle's formula row by row."""
import numpy as np
import torch

from oracle import attention as A


def random_parents(rng, n, roots=0.0, reach=8):
    """n rows: -1 for roots, else an earlier row at most `reach` back."""
    p = np.full(n, -1, dtype=np.int32)
    for r in range(1, n):
        if rng.random() >= roots:
            p[r] = rng.integers(max(0, r - reach), r)
    return p


def chain(parent, r):
    """Row r and its ancestors, from r on; a parent that is not below its row is none."""
    out = [r]
    while 0 <= parent[out[-1]] < out[-1]:
        out.append(int(parent[out[-1]]))
    return out


def ancestor_bits(parent, window=0, sinks=0, base=0):
    """(bits [n, n] truth values, depth [n])."""
    n = len(parent)
    bits, depth = np.zeros((n, n), dtype=bool), np.zeros(n, dtype=np.int64)
    for r in range(n):
        c = chain(parent, r)
        depth[r] = len(c) - 1
        for steps, a in enumerate(c):
            bits[r, a] = window == 0 or steps < window or base + depth[r] - steps < sinks
    return bits, depth


def words_of(bits, words):
    """int32 words of truth values [n, m]; columns past the words are dropped."""
    n = bits.shape[0]
    wide = np.zeros((n, words * 32), dtype=bool)
    m = min(bits.shape[1], words * 32)
    wide[:, :m] = bits[:, :m]
    return np.packbits(wide, axis=1, bitorder="little").view(np.uint32).reshape(n, words).view(np.int32)


def expect_tree(P, bits, positions, window=0, sinks=0, table=None, kv=None):
    """As Paged.expect, of rows that see the cached part by window and sinks and,
    of the new tokens, what bits[i] [n, n] of sequence i say."""
    scale = 1.0 / np.sqrt(P.d)
    table = P.table if table is None else table
    o = np.zeros((P.tokens, P.heads, P.d))
    tol, lse, ltol = np.zeros_like(o), np.zeros((P.tokens, P.heads)), np.zeros((P.tokens, P.heads))
    group = P.heads // P.kv_heads
    for i, (n, total) in enumerate(zip(P.news, P.totals)):
        k, v = (kv[0][i], kv[1][i]) if kv else (P.values(0, i), P.values(1, i))
        there = np.array([0 <= table[i, j // P.page] < P.pages for j in range(total)], dtype=bool)
        base, j = total - n, np.arange(total)
        for r in range(n):
            t = P.q_start[i] + r
            p = min(max(int(positions[t]), base), total - 1)
            see = (j < base) & ((window == 0) | (j > p - window) | (j < sinks))
            named = np.zeros(total, dtype=bool)
            first = max(0, -base)
            named[base + first:] = bits[i][r, first:n]
            see = (see | named) & there
            for h in range(P.heads):
                y, s, bound, logit = A.attend(P.q[t, h], k[:, h // group], v[:, h // group], see, scale)
                o[t, h], lse[t, h] = y, s
                tol[t, h] = A.tolerance(bound, logit, P.d)
                ltol[t, h] = 2.0 * (P.d / 8 + 8) * 2.0**-23 * logit + 2.0**-17 * max(1.0, abs(s) if np.isfinite(s) else 1.0)
    return o, tol, lse, ltol


def to_gpu(x, dev, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).to(dev)
