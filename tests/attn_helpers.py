"""Building paged caches and their expected results for the tests."""
import numpy as np
import torch

from oracle import attention as A


class Paged:
    """Sequences with `totals` cached tokens, of which the last `news` are the
    call's, in a shuffled pool built byte by byte from the oracle's packer."""

    def __init__(self, lq, fmt, news, totals, heads, kv_heads, d, page, dev, seed=0, scale_k=1.0, spare=2, fill="noise"):
        rng = np.random.default_rng(seed)
        self.lq, self.fmt, self.dev = lq, fmt, dev
        self.news, self.totals, self.heads, self.kv_heads, self.d, self.page = news, totals, heads, kv_heads, d, page
        self.tokens = int(sum(news))
        n = len(news)
        used = [-(-t // page) for t in totals]
        width = max(1, max(used))
        pages = sum(used) + spare
        order = rng.permutation(pages)
        self.table = np.full((n, width), -1, dtype=np.int32)
        at = 0
        for i, u in enumerate(used):
            self.table[i, :u] = order[at:at + u]
            at += u
        self.k = [(rng.standard_normal((t, kv_heads, d)) * scale_k).astype(np.float32) for t in totals]
        self.v = [rng.standard_normal((t, kv_heads, d)).astype(np.float32) for t in totals]
        self.q = rng.standard_normal((self.tokens, heads, d)).astype(np.float32)
        self.row = A.CODE_ROW[fmt](d)
        self.block = page * (self.row + (0 if fmt == "f16" else d // 16))
        noise = rng.integers(0, 256, size=(2, pages, kv_heads, self.block), dtype=np.uint8)
        if fill == "nan":  # slots that hold no token: all ones are NaN as f16
            noise[:] = 0xFF
        self.pools = noise
        for which, x in ((0, self.k), (1, self.v)):
            for i in range(n):
                self.store(which, i, x[i])
        self.q_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.pages = pages

    def store(self, which, i, x, first=0):
        """Rows x [m, kv_heads, D] at positions first .. of sequence i."""
        for h in range(self.kv_heads):
            if not len(x):
                continue
            codes, scales = A.cache_rows(self.fmt, x[:, h])
            for m in range(len(x)):
                pg, slot = self.table[i, (first + m) // self.page], (first + m) % self.page
                if pg < 0:
                    continue
                head = self.pools[which, pg, h]
                head[slot * self.row:(slot + 1) * self.row] = codes[m]
                if scales is not None:
                    at = self.page * self.row + slot * (self.d // 16)
                    head[at:at + self.d // 16] = scales[m].view(np.uint8)

    def cache(self):
        k, v = (torch.from_numpy(p.copy()).to(self.dev) for p in self.pools)
        return self.lq.KVCache(self.fmt, self.pages, self.page, self.kv_heads, self.d, k=k, v=v)

    def batch(self, max_q=0, table=None, kv_len=None, q_start=None):
        up = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(self.dev)  # noqa: E731
        return self.lq.KVBatch(up(self.table if table is None else table), up(self.totals if kv_len is None else kv_len),
                               up(self.q_start if q_start is None else q_start), self.tokens, max_q=max_q)

    def values(self, which, i):
        x = (self.k, self.v)[which][i]
        return A.cache_values(self.fmt, x.reshape(-1, self.d)).reshape(x.shape) if x.size else x

    def expect(self, window=0, sinks=0, scale=None, table=None, kv=None):
        """(o, tol, lse, lse tol) in float64; `kv`: values to use instead of
        the stored ones ((k, v) lists)."""
        scale = 1.0 / np.sqrt(self.d) if scale is None else scale
        table = self.table if table is None else table
        o = np.zeros((self.tokens, self.heads, self.d))
        tol, lse, ltol = np.zeros_like(o), np.zeros((self.tokens, self.heads)), np.zeros((self.tokens, self.heads))
        group = self.heads // self.kv_heads
        for i, (n, total) in enumerate(zip(self.news, self.totals)):
            k, v = (kv[0][i], kv[1][i]) if kv else (self.values(0, i), self.values(1, i))
            there = np.array([0 <= table[i, j // self.page] < self.pages for j in range(total)], dtype=bool)
            for r in range(n):
                see = A.visible(total - n + r, total, window, sinks) & there
                for h in range(self.heads):
                    t = self.q_start[i] + r
                    y, s, bound, logit = A.attend(self.q[t, h], k[:, h // group], v[:, h // group], see, scale)
                    o[t, h], lse[t, h] = y, s
                    tol[t, h] = A.tolerance(bound, logit, self.d)
                    ltol[t, h] = 2.0 * (self.d / 8 + 8) * 2.0**-23 * logit + 2.0**-17 * max(1.0, abs(s) if np.isfinite(s) else 1.0)
        return o, tol, lse, ltol


def compare(got, want, tol, what=""):
    got = np.asarray(got, dtype=np.float64)
    bad = ~(np.abs(got - want) <= tol) & ~(np.isnan(got) & np.isnan(want)) & (got != want)
    assert not bad.any(), (f"{what}: {np.count_nonzero(bad)} of {bad.size} outside tolerance; first at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]!r} against {want[bad][0]!r}, tolerance {tol[bad][0]:.3g}")
