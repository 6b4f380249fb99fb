"""The paged key/value cache and the attention over it: what is measured.

Three operators of a decoder's serving path, next to the projections that the
library already runs (f32 activations in, f32 out, weights in f16 / Q8_0 /
Q4_0):

* "write": the new tokens' keys and values are quantised into the pages of the
  cache (f16, Q8_0 or Q4_0), and the same tokens are read back as f32;
* "read": whole sequences are read back from the cache as f32;
* "attn": attention of each sequence's new tokens (one in decoding, a chunk in
  prefill) over its pages, causal, with shared key/value heads; with
  `window` > 0 only the last `window` positions stay visible, and the first
  `sinks` positions besides.

A pool holds, for every page and key/value head, the codes of `page` tokens
([page, head_dim], f16, int8, or 16 bytes a block of 32 with element j in the
low and element j + 16 in the high nibble of byte j) and then, for the
quantised formats, their f16 scales ([page, head_dim / 32]).
"""
import math

import numpy as np
import torch

own = False

_BITS = {"f16": 16.0, "q8_0": 8.5, "q4_0": 4.5}
_LIMIT = 65504.0  # the cache's range, in every format


# ---- cases ------------------------------------------------------------------
def _case(name, op, fmt, batch, new, kv, ragged, heads, kv_heads, head_dim, page, window=0, sinks=0):
    c = {"op": op, "fmt": fmt, "batch": batch, "new": new, "kv": kv, "ragged": ragged, "heads": heads,
         "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "window": window, "sinks": sinks}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decode step of eight sequences appends a token each: a latency
        _case("write_decode_q8_0", "write", "q8_0", 8, 1, 2000, True, 32, 8, 128, 16),
        # a long prompt enters a Q8_0 cache
        _case("write_prompt_q8_0", "write", "q8_0", 1, 16384, 16384, False, 32, 8, 128, 16),
        # several prompts of odd lengths enter a Q4_0 cache with wide heads
        _case("write_ragged_q4_0", "write", "q4_0", 7, 1999, 5000, True, 16, 2, 256, 64),
        # sequences leave a Q8_0 cache as f32 (another format, another host)
        _case("read_long_q8_0", "read", "q8_0", 4, 16001, 16001, True, 32, 8, 128, 32),
        # one token of one short sequence: the smallest call, a latency
        _case("decode_one_f16", "attn", "f16", 1, 1, 513, False, 32, 8, 128, 16),
        # a serving step: 64 sequences of mixed lengths, one token each
        _case("decode_batch_q8_0", "attn", "q8_0", 64, 1, 8192, True, 32, 8, 128, 16),
        # one very long sequence, wide heads, one token
        _case("decode_long_f16", "attn", "f16", 1, 1, 131071, False, 16, 2, 256, 64),
        # drafted tokens of 16 sequences are verified: four tokens each
        _case("verify_q4_0", "attn", "q4_0", 16, 4, 6000, True, 32, 8, 128, 32),
        # a chunk of a long prompt over the part that is cached already
        _case("chunk_q8_0", "attn", "q8_0", 1, 2048, 16384, False, 32, 8, 128, 16),
        # whole prompts of odd lengths, nothing cached before
        _case("prompts_f16", "attn", "f16", 3, 4001, 4001, True, 32, 8, 128, 16),
        # decoding with a sliding window and sinks over long sequences
        _case("window_decode_q8_0", "attn", "q8_0", 32, 1, 32768, True, 32, 4, 128, 64, 4096, 4),
        # a prompt under a sliding window with sinks, narrow heads
        _case("window_prompt_f16", "attn", "f16", 1, 8192, 8192, False, 32, 8, 64, 16, 1024, 4),
    ]


def draw(rng):
    """One more case of the listed ranges; its padded size and its work stay
    within the largest listed ones."""
    logint = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    while True:
        op = rng.choice(["write", "write", "read", "attn", "attn", "attn", "attn"])
        fmt = rng.choice(["f16", "q8_0", "q4_0"])
        kv_heads, head_dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        heads = kv_heads * rng.choice([1, 2, 4, 8])
        page = rng.choice([16, 16, 32, 64, 128])
        batch, kv = logint(1, 64), logint(17, 131071)
        window, sinks = 0, 0
        if op == "read":
            new = kv
        elif op == "write":
            new = logint(1, kv)
        else:
            new = rng.choice([1, 1, logint(1, 16), logint(16, 4001)])
            if rng.random() < 0.4:
                window, sinks = logint(16, 8192), rng.choice([0, 4, 4, 33])
        new = min(new, kv)
        case = _case(None, op, fmt, batch, new, kv, rng.random() < 0.6, heads, kv_heads, head_dim, page, window, sinks)
        if batch * kv * kv_heads * head_dim > 64 * 8192 * 8 * 128 or batch * heads * new * kv > 1 << 30 and op == "attn":
            continue  # the plain form's padded arrays
        cost = work(case)
        if cost["bytes"] <= (5e8 if op == "attn" else 3.4e8) and cost["flops"] <= 5e11:
            return case


def _lengths(case):
    """(new tokens, total length) of each sequence; a ragged batch spreads them
    over the case's ranges (the first sequence has the largest)."""
    b, new, kv = case["batch"], case["new"], case["kv"]
    if not case["ragged"]:
        return [new] * b, [kv] * b
    part = [1.0 - math.fmod(i * 0.6180339887498949, 1.0) for i in range(b)]
    news = [max(1, int(new * f)) for f in part]
    return news, [max(n, int(kv * math.fmod(f + 0.31 * i, 1.0)) if i else kv) for i, (n, f) in enumerate(zip(news, part))]


def _pairs(case):
    """Visible (query, key) pairs of one head, and the keys that any of a
    sequence's new tokens sees, both summed over the sequences."""
    pairs = keys = 0
    w, s = case["window"], case["sinks"]
    for n, total in zip(*_lengths(case)):
        pos = np.arange(total - n, total, dtype=np.int64)
        seen = pos + 1
        if w:
            seen = np.where(seen > w, w + np.minimum(s, np.maximum(seen - w, 0)), seen)
        pairs += int(seen.sum())
        keys += min(total, n + w - 1 + s) if w else total
    return pairs, keys


def work(case):
    news, totals = _lengths(case)
    tokens, d = sum(news), case["head_dim"]
    packed = 2 * case["kv_heads"] * d * _BITS[case["fmt"]] / 8  # K and V of one token in the cache
    plain = 2 * case["kv_heads"] * d * 4
    if case["op"] == "write":
        return {"bytes": tokens * 2 * (plain + packed), "flops": tokens * 8 * case["kv_heads"] * d}
    if case["op"] == "read":
        return {"bytes": tokens * (plain + packed), "flops": tokens * 2 * case["kv_heads"] * d}
    pairs, keys = _pairs(case)
    return {"bytes": keys * packed + 2 * tokens * case["heads"] * d * 4, "flops": 4 * pairs * case["heads"] * d}


# ---- inputs -----------------------------------------------------------------
def _quantise(x, fmt):
    """x [..., D] f32 -> (codes, scales) as the pool holds them: int8 / uint8
    codes and f16 scales, by the rules of the weight formats."""
    x = x.clamp(-_LIMIT, _LIMIT)
    if fmt == "f16":
        return x.to(torch.float16), None
    b = x.unflatten(-1, (-1, 32))
    size = b.abs()
    top = size.amax(-1, keepdim=True)
    if fmt == "q8_0":
        d = top / torch.full_like(top, 127.0)
        y = b / torch.where(d == 0, 1.0, d)
        q = y.trunc()
        q = q + torch.where((y - q).abs() >= 0.5, torch.sign(y), 0.0)
        q = torch.where(d == 0, 0.0, q.clamp(-127, 127)).to(torch.int8)
        return q.flatten(-2), d.squeeze(-1).to(torch.float16)
    first = torch.where(size == top, torch.arange(32, device=x.device), 32).amin(-1, keepdim=True)
    d = b.gather(-1, first) / torch.full_like(top, -8.0)
    q = (b / torch.where(d == 0, 1.0, d) + 8.5).to(torch.int32).clamp(0, 15)
    q = torch.where(d == 0, 8, q).to(torch.uint8)
    return (q[..., :16] | (q[..., 16:] << 4)).flatten(-2), d.squeeze(-1).to(torch.float16)


def _values(codes, scales, fmt):
    """The f32 values that codes and scales stand for."""
    if fmt == "f16":
        return codes.to(torch.float32)
    if fmt == "q8_0":
        q = codes.to(torch.float32).unflatten(-1, (-1, 32))
    else:
        b = codes.unflatten(-1, (-1, 16))
        q = torch.cat([b & 15, b >> 4], -1).to(torch.float32) - 8.0
    return (q * scales.to(torch.float32).unsqueeze(-1)).flatten(-2)


def _parts(pool, case):
    """(codes, scales) views of a pool [pages, kv_heads, bytes]."""
    fmt, page, d = case["fmt"], case["page"], case["head_dim"]
    if fmt == "f16":
        return pool.view(torch.float16).unflatten(-1, (page, d)), None
    row = d if fmt == "q8_0" else d // 2
    codes = pool[..., : page * row].unflatten(-1, (page, row))
    return codes.view(torch.int8) if fmt == "q8_0" else codes, pool[..., page * row:].view(torch.float16).unflatten(-1, (page, d // 32))


def _tokens(g, rows, heads, d, spread, dev):
    """Keys, values or queries: normal, each channel with a size of its own."""
    size = torch.exp(spread * torch.randn(heads, d, generator=g, device=dev))
    return torch.randn(rows, heads, d, generator=g, device=dev) * size


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    news, totals = _lengths(case)
    b, d, page, hkv = case["batch"], case["head_dim"], case["page"], case["kv_heads"]
    width = -(-max(totals) // page)
    used = [-(-t // page) for t in totals]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = np.full((b, width), -1, dtype=np.int64)
    start = 0
    for i, n in enumerate(used):
        table[i, :n] = np.arange(start, start + n)
        start += n
    table = torch.from_numpy(table).to(dev)
    table = torch.where(table >= 0, order[table.clamp(min=0)], -1).to(torch.int32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=dev)
    s = {"case": dict(case), "table": table, "kv_len": torch.tensor(totals, dtype=torch.int32, device=dev), "q_start": cu,
         "tokens": sum(news), "max_new": max(news), "max_kv": max(totals), "pages": pages, "handles": None}
    for name in ("k", "v"):
        spread = 0.5 if name == "k" else 0.2
        block = int(page * d * _BITS[case["fmt"]] / 8)
        pool = torch.zeros(pages, hkv, block, dtype=torch.uint8, device=dev)
        if case["op"] != "write":
            codes, scales = _parts(pool, case)
            step = max(1, (1 << 26) // (hkv * page * d))
            size = torch.exp(spread * torch.randn(hkv, 1, d, generator=g, device=dev))
            for p in range(0, pages, step):
                n = min(step, pages - p)
                c, sc = _quantise(torch.randn(n, hkv, page, d, generator=g, device=dev) * size, case["fmt"])
                codes[p:p + n] = c
                if sc is not None:
                    scales[p:p + n] = sc
        else:
            s["new_" + name] = _tokens(g, s["tokens"], hkv, d, spread, dev)
        s["pool_" + name] = pool
        s["out_" + name] = torch.empty(s["tokens"], hkv, d, device=dev) if case["op"] != "attn" else None
    if case["op"] == "attn":
        s["q"] = _tokens(g, s["tokens"], case["heads"], d, 0.3, dev)
        s["out"] = torch.empty_like(s["q"])
    return s


# ---- one pass ---------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import gemm_gemv_f16w_gb300 as lq

    case = state["case"]
    if state["handles"] is None:  # what a server makes once: the cache, the step's batch, the scratch memory
        cache = lq.KVCache(case["fmt"], state["pages"], case["page"], case["kv_heads"], case["head_dim"],
                           k=state["pool_k"], v=state["pool_v"])
        batch = lq.KVBatch(state["table"], state["kv_len"], state["q_start"], state["tokens"], max_q=state["max_new"])
        work = lq.attn_work(cache, batch, case["heads"]) if case["op"] == "attn" else None
        state["handles"] = cache, batch, work
    cache, batch, work = state["handles"]
    if case["op"] == "attn":
        lq.lq_attn_paged(cache, batch, state["q"], state["out"], 1.0 / math.sqrt(case["head_dim"]),
                         window=case["window"], sinks=case["sinks"], work=work)
        return state["out"]
    if case["op"] == "write":
        lq.lq_kv_write(cache, batch, state["new_k"], state["new_v"])
    lq.lq_kv_read(cache, batch, state["out_k"], state["out_v"])
    return state["out_k"], state["out_v"]


def _places(state):
    """Sequence, position, page and slot of every new token."""
    page = state["case"]["page"]
    t = torch.arange(state["tokens"], device=state["table"].device)
    seq = torch.searchsorted(state["q_start"].long(), t, right=True) - 1
    pos = state["kv_len"].long()[seq] - state["q_start"].long()[seq + 1] + t
    return seq, pos, state["table"].long()[seq, pos // page], pos % page


def _run_plain(state):
    case = state["case"]
    fmt, d, hkv = case["fmt"], case["head_dim"], case["kv_heads"]
    seq, pos, at, slot = _places(state)
    codes_k, scales_k = _parts(state["pool_k"], case)
    codes_v, scales_v = _parts(state["pool_v"], case)
    if case["op"] != "attn":
        if case["op"] == "write":
            k, dk = _quantise(state["new_k"], fmt)
            v, dv = _quantise(state["new_v"], fmt)
            codes_k[at, :, slot], codes_v[at, :, slot] = k, v
            if fmt != "f16":
                scales_k[at, :, slot], scales_v[at, :, slot] = dk, dv
        pick = lambda x: None if x is None else x[at, :, slot]  # noqa: E731
        return _values(pick(codes_k), pick(scales_k), fmt), _values(pick(codes_v), pick(scales_v), fmt)
    # every sequence padded to the longest: [batch, kv_heads, keys, head_dim]
    b, most, new, group = case["batch"], state["table"].shape[1] * case["page"], state["max_new"], case["heads"] // hkv
    table = state["table"].long().clamp(min=0)
    lay = lambda c, s: _values(c[table], None if s is None else s[table], fmt).transpose(1, 2).reshape(b, hkv, most, d)  # noqa: E731
    row = torch.arange(state["tokens"], device=seq.device) - state["q_start"].long()[seq]
    q = torch.zeros(b, new, case["heads"], d, device=seq.device)
    q[seq, row] = state["q"] * (1.0 / math.sqrt(d))
    q = q.view(b, new, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * new, d)
    scores = (q @ lay(codes_k, scales_k).transpose(-1, -2)).view(b, hkv, group, new, most)
    first = (state["kv_len"] - state["q_start"][1:] + state["q_start"][:-1]).long()
    p, j = (first[:, None] + torch.arange(new, device=seq.device))[..., None], torch.arange(most, device=seq.device)
    hidden = j > p
    if case["window"]:
        hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    scores = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = scores.view(b, hkv, group * new, most) @ lay(codes_v, scales_v)
    out = out.view(b, hkv, group, new, d) / total
    return out.permute(0, 3, 1, 2, 4).reshape(b, new, case["heads"], d)[seq, row]


# ---- the definition, in 64 bits ---------------------------------------------
def exact(case, seed):
    """Sequence by sequence and head by head in float64. The quantisers' rules
    hold the scale and the quotients as float32, which is restated here from
    float64 values (a quotient of two float32 numbers rounded to float64 and
    then to float32 is the float32 quotient)."""
    if case["op"] == "attn" and 4.0 * _pairs(case)[0] * case["heads"] * case["head_dim"] > 4e12:
        return None
    s = prepare(case, seed)
    news, totals = _lengths(case)
    fmt, d, page = case["fmt"], case["head_dim"], case["page"]
    f64 = torch.float64

    def stored(x):  # values that the cache keeps of x [n, D]
        x = x.to(f64).clamp(-_LIMIT, _LIMIT)
        if fmt == "f16":
            return x.to(torch.float32).to(torch.float16).to(f64)
        r32 = lambda y: y.to(torch.float32).to(f64)  # noqa: E731
        b = x.reshape(-1, 32)
        rows = torch.arange(b.shape[0], device=b.device)
        if fmt == "q8_0":
            scale = r32(b.abs().max(1).values / 127.0)
            y = r32(b / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None])
            code = torch.copysign(torch.floor(y.abs() + 0.5), y).clamp(-127, 127)
        else:
            lead = ((b.abs() == b.abs().amax(1, keepdim=True)).cumsum(1) == 0).sum(1)  # the first of the largest
            scale = r32(b[rows, lead] / -8.0)
            y = r32(r32(b / torch.where(scale != 0, scale, torch.ones_like(scale))[:, None]) + 8.5)
            code = torch.floor(y).clamp(0, 15) - 8.0
        code = torch.where((scale != 0)[:, None], code, torch.zeros_like(code))
        return (code * scale.to(torch.float32).to(torch.float16).to(f64)[:, None]).reshape(x.shape)

    def kept(pool, i, h, n):  # the first n positions of sequence i, head h, from the pool's bytes
        ids = s["table"][i, : -(-n // page)].long()
        raw = pool[ids, h]
        if fmt == "f16":
            return raw.contiguous().view(torch.float16).reshape(-1, d)[:n].to(f64)
        row = d if fmt == "q8_0" else d // 2
        scale = raw[:, page * row:].contiguous().view(torch.float16).reshape(-1, d // 32)[:n].to(f64)
        c = raw[:, : page * row].reshape(-1, row)[:n]
        if fmt == "q8_0":
            c = c.contiguous().view(torch.int8).to(f64)
        else:
            c = c.reshape(n, d // 32, 16).to(torch.int32)
            c = torch.stack([c % 16, c // 16], 2).reshape(n, d).to(f64) - 8.0
        return c * scale.repeat_interleave(32, 1)

    if case["op"] == "write":
        return stored(s["new_k"]), stored(s["new_v"])
    if case["op"] == "read":
        outs = []
        for pool in (s["pool_k"], s["pool_v"]):
            outs.append(torch.cat([torch.stack([kept(pool, i, h, totals[i])[totals[i] - n:] for h in range(case["kv_heads"])], 1)
                                   for i, n in enumerate(news)]))
        return tuple(outs)
    out = torch.empty(s["tokens"], case["heads"], d, dtype=f64, device=s["q"].device)
    group, at = case["heads"] // case["kv_heads"], 0
    for i, n in enumerate(news):
        for h in range(case["kv_heads"]):
            k, v = kept(s["pool_k"], i, h, totals[i]), kept(s["pool_v"], i, h, totals[i])
            for r in range(0, n, 1024):
                rows = min(1024, n - r)
                pos = torch.arange(totals[i] - n + r, totals[i] - n + r + rows, device=k.device)[:, None]
                j = torch.arange(totals[i], device=k.device)[None]
                see = j <= pos
                if case["window"]:
                    see &= (j > pos - case["window"]) | (j < case["sinks"])
                q = s["q"][at + r: at + r + rows, h * group: (h + 1) * group].to(f64)
                x = torch.einsum("tgd,kd->gtk", q, k) / math.sqrt(d)
                w = torch.softmax(torch.where(see, x, torch.full_like(x, -math.inf)), -1)
                out[at + r: at + r + rows, h * group: (h + 1) * group] = torch.einsum("gtk,kd->tgd", w, v)
        at += n
    return out
