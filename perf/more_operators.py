"""Drafted tokens, beams and rotary positions around the paged cache: what is
measured.

Five operators of a decoder's serving path, next to the cache and the attention
that the library already has (f32 activations in, f32 out, a cache in f16, Q8_0
or Q4_0):

* "rope": rotary positions of one to three axes (time, height, width) turn the
  queries and keys of a fused projection's rows, whole heads or a part of them;
* "tree": attention of a tree of drafted tokens over each sequence's pages: all
  of what was cached before, and of the new tokens those that a row's bits name
  (its ancestors and itself);
* "draft": what a verified draft needs besides: every row's position and bits
  from the tree's parents, the longest path that the model's own choices
  confirm, and that path's keys and values moved to the places where the
  cache goes on;
* "beams": beam search's selection, the best of all beams' continuations by
  score + log softmax(logits);
* "states": the beams' page tables follow their parents, and the last, partly
  filled pages are copied where several beams go on from one.

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


# ---- cases ------------------------------------------------------------------
def _rope(name, tokens, heads, kv_heads, head_dim, rotary, axes, turns, adjacent, base, far):
    c = {"op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "rotary": rotary,
         "axes": axes, "turns": turns, "adjacent": adjacent, "base": base, "far": far}
    return {"name": name, **c} if name else c


def _tree(name, fmt, batch, new, kv, ragged, heads, kv_heads, head_dim, page, window=0, sinks=0):
    c = {"op": "tree", "fmt": fmt, "batch": batch, "new": new, "kv": kv, "ragged": ragged, "heads": heads,
         "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "window": window, "sinks": sinks}
    return {"name": name, **c} if name else c


def _draft(name, fmt, batch, new, kv, kv_heads, head_dim, page):
    c = {"op": "draft", "fmt": fmt, "batch": batch, "new": new, "kv": kv, "ragged": batch > 1, "kv_heads": kv_heads,
         "head_dim": head_dim, "page": page}
    return {"name": name, **c} if name else c


def _beams(name, groups, beams, vocab, keep, first, ended, coarse):
    c = {"op": "beams", "groups": groups, "beams": beams, "vocab": vocab, "keep": keep, "first": first, "ended": ended,
         "coarse": coarse}
    return {"name": name, **c} if name else c


def _states(name, fmt, groups, beams, kv, kv_heads, head_dim, page):
    c = {"op": "states", "fmt": fmt, "groups": groups, "beams": beams, "kv": kv, "kv_heads": kv_heads,
         "head_dim": head_dim, "page": page}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decode step of 32 sequences far into their contexts: a latency
        _rope("rope_step", 32, 32, 8, 128, 128, 1, False, False, 1e6, 131071),
        # a long prompt of a video's patches: three axes that take turns over the pairs of a head, an odd count
        _rope("rope_patches", 16383, 32, 8, 128, 128, 3, True, False, 5e6, 2000),
        # one sequence, a small tree: a latency
        _tree("tree_one_f16", "f16", 1, 7, 2000, False, 32, 8, 128, 16),
        # a serving step: every sequence has a few branches to verify
        _tree("tree_step_q8_0", "q8_0", 32, 12, 6000, True, 32, 8, 128, 16),
        # wide trees of odd sizes
        _tree("tree_wide_f16", "f16", 16, 61, 8192, True, 32, 8, 128, 32),
        # a window with sinks, wide heads, the smallest cache
        _tree("tree_window_q4_0", "q4_0", 8, 33, 32768, True, 16, 2, 256, 64, 4096, 4),
        # bookkeeping of one sequence's small tree: a latency
        _draft("draft_one_f16", "f16", 1, 7, 2000, 8, 128, 16),
        # bookkeeping of a step: 32 sequences, trees of up to 61 rows
        _draft("draft_step_q8_0", "q8_0", 32, 61, 4000, 8, 128, 16),
        # one sequence, four beams: a latency
        _beams("beams_one", 1, 4, 151936, 8, False, False, False),
        # a batch of beam searches, some beams ended, logits of a coarse head (ties)
        _beams("beams_batch", 32, 8, 151936, 16, False, True, True),
        # one search moves on
        _states("states_one_f16", "f16", 1, 4, 1000, 8, 128, 16),
        # many searches move on, large pages
        _states("states_batch_f16", "f16", 64, 8, 1900, 8, 128, 128),
    ]


def draw(rng):
    """One more case of the listed ranges; its padded size and its work stay
    within the largest listed ones."""
    logint = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    while True:
        op = rng.choice(["rope", "rope", "tree", "tree", "tree", "tree", "draft", "beams", "beams", "states"])
        fmt = rng.choice(["f16", "q8_0", "q4_0"])
        kv_heads, head_dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256]), rng.choice([16, 16, 32, 64, 128])
        heads = kv_heads * rng.choice([1, 2, 4, 8])
        if op == "rope":
            axes, rotary = rng.choice([1, 1, 2, 3]), rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
            case = _rope(None, logint(1, 16383), heads, kv_heads, head_dim, rotary, axes, axes > 1 and rng.random() < 0.5,
                         rng.random() < 0.3, rng.choice([1e4, 5e5, 1e6, 1e7]), rng.choice([0, 2000, 131071, 1000003]))
            if work(case)["bytes"] > 6.8e8:
                continue
        elif op == "tree":
            batch, kv, new = logint(1, 64), logint(17, 65536), logint(1, 200)
            window, sinks = (logint(16, 8192), rng.choice([0, 4, 4, 33])) if rng.random() < 0.3 else (0, 0)
            case = _tree(None, fmt, batch, min(new, kv), kv, rng.random() < 0.6, heads, kv_heads, head_dim, page, window, sinks)
            cost = work(case)
            # (the plain form's padded arrays)
            if batch * kv * kv_heads * head_dim > 1 << 28 or batch * heads * new * kv > 1 << 28 or cost["bytes"] > 2.8e8 or cost["flops"] > 6e10:
                continue
        elif op == "draft":
            batch, new = logint(1, 64), logint(2, 100)
            case = _draft(None, fmt, batch, new, max(new, logint(17, 8192)), kv_heads, head_dim, page)
            if batch * new > 3000 or work(case)["bytes"] > 2.5e7 or batch * case["kv"] * kv_heads * head_dim > 1 << 28:
                continue
        elif op == "beams":
            beams = rng.choice([2, 3, 4, 5, 8, 16])
            case = _beams(None, logint(1, 64), beams, rng.choice([151936, logint(500, 151936), logint(500, 151936)]),
                          rng.choice([beams, 2 * beams]), rng.random() < 0.2, rng.random() < 0.3, rng.random() < 0.4)
            if case["groups"] * beams * case["vocab"] > 32 * 8 * 151936:
                continue
        else:
            case = _states(None, fmt, logint(1, 64), rng.choice([2, 3, 4, 5, 8, 16]), logint(17, 4000), kv_heads, head_dim, page)
            if case["groups"] * case["beams"] * page * kv_heads * head_dim > 64 * 8 * 128 * 8 * 128:
                continue
            if case["groups"] * (case["beams"] * page + case["kv"]) * kv_heads * head_dim > 64 * (8 * 128 + 1900) * 8 * 128:
                continue
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


def _token_bytes(case):
    """K and V of one token in the cache."""
    return 2 * case["kv_heads"] * case["head_dim"] * _BITS[case["fmt"]] / 8


def work(case):
    op = case["op"]
    if op == "rope":
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["head_dim"]
        return {"bytes": 8 * values + 4 * case["axes"] * case["tokens"],
                "flops": 3 * case["tokens"] * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    if op == "beams":
        rows, v = case["groups"] * case["beams"], case["vocab"]
        return {"bytes": 4 * rows * v + 8 * rows + 12 * case["groups"] * case["keep"], "flops": 4 * rows * v}
    if op == "states":
        rows, n = case["kv"] % case["page"], case["groups"] * case["beams"]
        # random parents: of n beams (1 - 1/n)^n, about 1/e, have no child and take another's copy
        copies = n * (1.0 - 1.0 / case["beams"]) ** case["beams"]
        return {"bytes": 2 * copies * rows * _token_bytes(case) + 8 * n * (-(-case["kv"] // case["page"]) + 3), "flops": 0}
    news, totals = _lengths(case)
    tokens = sum(news)
    if op == "draft":
        words = -(-max(news) // 32)
        # about four accepted rows of a sequence move
        return {"bytes": 2 * 4 * case["batch"] * _token_bytes(case) + tokens * (16 + 4 * words), "flops": 0}
    pairs = keys = 0
    for n, total in zip(news, totals):
        before = total - n
        if case["window"]:
            before = min(before, case["window"] + case["sinks"])
        keys += before + n
        pairs += n * before + n * min(n, 5)  # (a row has about four ancestors)
    return {"bytes": keys * _token_bytes(case) + 2 * tokens * case["heads"] * case["head_dim"] * 4,
            "flops": 4 * pairs * case["heads"] * case["head_dim"]}


# ---- inputs -----------------------------------------------------------------
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


def _pool(g, case, pages, spread, dev):
    """A pool full of normal values, each channel with a size of its own."""
    fmt, page, d, hkv = case["fmt"], case["page"], case["head_dim"], case["kv_heads"]
    pool = torch.zeros(pages, hkv, int(page * d * _BITS[fmt] / 8), dtype=torch.uint8, device=dev)
    codes, scales = _parts(pool, case)
    size = torch.exp(spread * torch.randn(hkv, 1, d, generator=g, device=dev))
    step = max(1, (1 << 26) // (hkv * page * d))
    for p in range(0, pages, step):
        x = torch.randn(min(step, pages - p), hkv, page, d, generator=g, device=dev) * size
        if fmt == "f16":
            codes[p:p + step] = x.to(torch.float16)
            continue
        x = x.unflatten(-1, (-1, 32))
        top = x.abs().amax(-1, keepdim=True) / (127.0 if fmt == "q8_0" else 7.0)
        q = torch.round(x / top.clamp(min=1e-30)).to(torch.int32)
        if fmt == "q8_0":
            codes[p:p + step] = q.to(torch.int8).flatten(-2)
        else:
            q = (q + 8).to(torch.uint8)
            codes[p:p + step] = (q[..., :16] | (q[..., 16:] << 4)).flatten(-2)
        scales[p:p + step] = top.squeeze(-1).to(torch.float16)
    return pool


def _trees(g, news, dev):
    """Parents of every row: row 0 is a sequence's root, another row's parent
    is one of the eight rows before it."""
    at = torch.cat([torch.arange(n) for n in news]).to(dev)
    back = 1 + (torch.rand(at.numel(), generator=g, device=dev) * torch.clamp(at, max=8)).long()
    return torch.where(at > 0, torch.clamp(at - back, min=0), -1).to(torch.int32)


def _padded(case, q_start, x, fill):
    """Rows x [tokens] as [batch, new], `fill` where a sequence has fewer."""
    at = q_start[:-1, None].long() + torch.arange(case["new"], device=x.device)
    there = at < q_start[1:, None]
    return torch.where(there, x[at.clamp(max=x.numel() - 1)], fill), there


def _ancestors(parent):
    """[batch, new, new] truth values: column a is row r's ancestor, or r."""
    b, n = parent.shape
    rows = torch.arange(n, device=parent.device)
    link = ((parent[..., None] == rows) & (parent[..., None] < rows[:, None])).float() + torch.eye(n, device=parent.device)
    for _ in range(max(1, (n - 1).bit_length())):
        link = (link @ link > 0).float()
    return link > 0


def _words(bits, words):
    """Truth values [..., n] as int32 words of 32, the first in the lowest bit."""
    pad = torch.nn.functional.pad(bits.long(), (0, words * 32 - bits.shape[-1])).unflatten(-1, (words, 32))
    return (pad << torch.arange(32, device=bits.device)).sum(-1).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    randn = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    s = {"case": dict(case), "handles": None}
    op = case["op"]
    if op == "rope":
        t, h, hkv, d, axes = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], case["axes"]
        rows = randn(t, (h + 2 * hkv) * d)  # a fused projection's output
        s["q"], s["k"] = rows[:, : h * d].unflatten(1, (h, d)), rows[:, h * d: (h + hkv) * d].unflatten(1, (hkv, d))
        s["q_out"], s["k_out"] = torch.empty(t, h, d, device=dev), torch.empty(t, hkv, d, device=dev)
        i, side = torch.arange(t, device=dev), math.isqrt(max(t // 4, 1)) + 1
        start = torch.randint(0, case["far"] + 1, (1,), generator=g, device=dev)
        if t <= 64:  # a step: every token is another sequence's
            pos = torch.randint(0, case["far"] + 1, (axes, t), generator=g, device=dev)
        else:
            pos = start + torch.stack([i, i, i] if axes == 1 else [i // (side * side), i // side % side, i % side])[:axes]
        s["pos"] = pos.to(torch.int32).contiguous()
        half = case["rotary"] // 2
        part = half // axes
        s["sections"] = [half - part * (axes - 1)] + [part] * (axes - 1)
        return s
    if op == "beams":
        n, v = case["groups"] * case["beams"], case["vocab"]
        x = 2.5 * randn(n, v)
        s["logits"] = torch.round(x * 16) / 16 if case["coarse"] else x
        scores = -20.0 * torch.rand(n, generator=g, device=dev)
        late = torch.arange(n, device=dev) % case["beams"] > 0
        s["scores"] = torch.where(late, -math.inf, 0.0) if case["first"] else scores
        s["ended"] = (torch.rand(n, generator=g, device=dev) < 0.2).to(torch.int32) if case["ended"] else None
        return s
    if op == "states":
        b, n, kv, page = case["groups"], case["beams"], case["kv"], case["page"]
        full, tail = kv // page, 2  # the last pages of a beam are its own
        pages = b * (full + n * tail)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(b, full + n * tail)
        table = torch.cat([order[:, None, :full].expand(b, n, full), order[:, full:].view(b, n, tail)], 2)
        s["table"] = table.reshape(b * n, full + tail).contiguous()
        s["parent"] = torch.randint(0, n, (b * n,), generator=g, device=dev).to(torch.int32)
        s["kv_len"] = torch.full((b * n,), kv, dtype=torch.int32, device=dev)
        s["pages"] = pages
        block = int(page * case["head_dim"] * _BITS[case["fmt"]] / 8)
        for name in ("k", "v"):  # (bytes are moved, whatever they stand for)
            s["pool_" + name] = torch.randint(0, 256, (pages, case["kv_heads"], block), generator=g, device=dev, dtype=torch.uint8)
        return s
    news, totals = _lengths(case)
    b, page = case["batch"], case["page"]
    width, used = -(-max(totals) // page), [-(-t // page) for t in totals]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = np.full((b, width), -1, dtype=np.int64)
    start = 0
    for i, n in enumerate(used):
        table[i, :n] = np.arange(start, start + n)
        start += n
    table = torch.from_numpy(table).to(dev)
    s["table"] = torch.where(table >= 0, order[table.clamp(min=0)], -1).to(torch.int32)
    s["kv_len"] = torch.tensor(totals, dtype=torch.int32, device=dev)
    s["q_start"] = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=dev)
    s |= {"tokens": sum(news), "max_new": max(news), "pages": pages}
    s["pool_k"], s["pool_v"] = _pool(g, case, pages, 0.5, dev), _pool(g, case, pages, 0.2, dev)
    s["parent"] = _trees(g, news, dev)
    words = -(-max(news) // 32)
    if op == "draft":
        s["token"] = torch.randint(0, 151936, (s["tokens"],), generator=g, device=dev).to(torch.int32)
        # the model's choice after a row: mostly the token of one of its children
        row = torch.arange(s["tokens"], device=dev)
        first = s["q_start"].long()[torch.searchsorted(s["q_start"].long(), row, right=True) - 1]
        above = torch.where(s["parent"] >= 0, first + s["parent"], s["tokens"])
        child = torch.full((s["tokens"] + 1,), -1, dtype=torch.long, device=dev).scatter_reduce(0, above, row, "amax")[:-1]
        agrees = (torch.rand(s["tokens"], generator=g, device=dev) < 0.85) & (child >= 0)
        other = torch.randint(0, 151936, (s["tokens"],), generator=g, device=dev).to(torch.int32)
        s["target"] = torch.where(agrees, s["token"][child.clamp(min=0)], other)
        s["most"] = 16
        return s
    # what the step's other part has left: positions and bits of every row
    parent, there = _padded(case, s["q_start"], s["parent"], -1)
    above = _ancestors(parent)
    base = s["kv_len"] - s["q_start"][1:] + s["q_start"][:-1]
    s["pos"] = (base[:, None] + above.sum(-1) - 1)[there].to(torch.int32)
    s["mask"] = _words(above, words)[there].contiguous()
    size = torch.exp(0.3 * randn(case["heads"], case["head_dim"]))
    s["q"] = randn(s["tokens"], case["heads"], case["head_dim"]) * size
    s["out"] = torch.empty_like(s["q"])
    return s


# ---- one pass ---------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import gemm_gemv_f16w_gb300 as lq

    case, op, made = state["case"], state["case"]["op"], state["handles"]
    if op == "rope":
        if made is None:  # what a model makes once
            made = state["handles"] = lq.Rope(case["head_dim"], case["rotary"], base=case["base"], adjacent=case["adjacent"],
                                              sections=state["sections"], interleaved=case["turns"])
        lq.lq_rope(made, state["pos"], state["q"], state["k"], q_out=state["q_out"], k_out=state["k_out"])
        return state["q_out"], state["k_out"]
    if op == "beams":
        if made is None:  # results and scratch memory of a search
            made = state["handles"] = lq.beam_buffers(case["groups"], case["beams"], case["vocab"], case["keep"])
        scores, parent, token, work = made
        lq.lq_beam_select(state["logits"], state["scores"], case["beams"], case["keep"], scores, parent, token, work,
                          finished=state["ended"], pad=0)
        return scores, parent, token
    if made is None:  # the cache, the step's batch, the buffers that a server keeps
        cache = lq.KVCache(case["fmt"], state["pages"], case["page"], case["kv_heads"], case["head_dim"],
                           k=state["pool_k"], v=state["pool_v"])
        ints = lambda *shape: torch.empty(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
        if op == "states":
            made = cache, torch.empty_like(state["table"]), ints(state["table"].shape[0], 3)
        else:
            batch = lq.KVBatch(state["table"], state["kv_len"], state["q_start"], state["tokens"], max_q=state["max_new"])
            if op == "tree":
                made = cache, batch, lq.attn_work(cache, batch, case["heads"])
            else:
                b, t = case["batch"], state["tokens"]
                made = cache, batch, ints(t), ints(t, -(-state["max_new"] // 32)), ints(b, state["most"]), ints(b), ints(b), ints(b)
        state["handles"] = made
    if op == "states":
        cache, table, copies = made
        lq.lq_beam_pages(state["parent"], case["beams"], state["table"], state["kv_len"], case["page"], table, copies)
        lq.lq_kv_copy(cache, copies)
        return table, copies, state["pool_k"], state["pool_v"]
    if op == "tree":
        cache, batch, work = made
        lq.lq_attn_tree(cache, batch, state["mask"], state["q"], state["out"], 1.0 / math.sqrt(case["head_dim"]),
                        positions=state["pos"], window=case["window"], sinks=case["sinks"], work=work)
        return state["out"]
    cache, batch, pos, mask, keep, count, token, length = made
    lq.lq_tree_plan(batch, state["parent"], pos, mask)
    lq.lq_tree_accept(batch, state["parent"], state["token"], state["target"], keep, count, token, length)
    lq.lq_kv_keep(cache, batch, keep, count)
    return pos, mask, keep, count, token, length, state["pool_k"], state["pool_v"]


def _run_plain(state):
    return {"rope": _plain_rope, "beams": _plain_beams, "states": _plain_states, "tree": _plain_tree, "draft": _plain_draft}[state["case"]["op"]](state)


def _pair_axes(case, sections):
    """The axis of every pair: sections one after another, or in turns."""
    half, axes = case["rotary"] // 2, case["axes"]
    j = torch.arange(half, device="cuda")
    size = torch.tensor(sections, device="cuda")
    if case["turns"]:
        return torch.where(j < axes * size[j % axes], j % axes, 0)
    return torch.searchsorted(size.cumsum(0), j, right=True)


def _plain_rope(state):
    case, half = state["case"], state["case"]["rotary"] // 2
    freq = torch.pow(torch.tensor(case["base"], dtype=torch.float64, device="cuda"),
                     torch.arange(half, dtype=torch.float64, device="cuda") * (-2.0 / case["rotary"]))
    angle = state["pos"].double()[_pair_axes(case, state["sections"])].t() * freq  # [tokens, half]: far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x):
        y = x.clone()
        if case["adjacent"]:
            a, b = x[..., 0: 2 * half: 2], x[..., 1: 2 * half: 2]
            y[..., 0: 2 * half: 2], y[..., 1: 2 * half: 2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :half], x[..., half: 2 * half]
            y[..., :half], y[..., half: 2 * half] = a * cos - b * sin, b * cos + a * sin
        return y

    return turned(state["q"]), turned(state["k"])


def _plain_beams(state):
    case = state["case"]
    n, v, keep = case["beams"], case["vocab"], case["keep"]
    x = state["logits"].double()  # values next to a border: the order has to be right
    top = x.amax(1, keepdim=True)
    score = x - top
    score = state["scores"].double()[:, None] + (score - torch.log(torch.exp(score).sum(1, keepdim=True)))
    if state["ended"] is not None:  # an ended beam stays as it is, with the padding token
        ended = state["ended"].bool()[:, None]
        stays = torch.where(torch.arange(v, device=x.device) == 0, state["scores"].double()[:, None], -math.inf)
        score = torch.where(ended, stays, score)
    score = torch.where(torch.isnan(score), -math.inf, score).view(case["groups"], n * v)
    best, at = torch.sort(score, dim=1, descending=True, stable=True)
    best, at = best[:, :keep], at[:, :keep]
    none = best == -math.inf
    return best.float(), torch.where(none, -1, at // v).to(torch.int32), torch.where(none, -1, at % v).to(torch.int32)


def _plain_states(state):
    case, table = state["case"], state["table"]
    b, n, page = case["groups"], case["beams"], case["page"]
    parent = state["parent"].view(b, n).long()
    i = torch.arange(n, device=parent.device)
    valid = (parent >= 0) & (parent < n)
    again = ((parent[:, :, None] == parent[:, None, :]) & (i[None, :] < i[:, None])).any(2)  # an earlier beam has the same parent
    extra = ~valid | again
    childless = ~(parent[:, None, :] == i[:, None]).any(2)
    # the m-th beam that cannot go on in its parent's pages takes those of the m-th beam without a child
    free = torch.argsort((~childless).to(torch.int32), dim=1, stable=True)
    place = torch.where(extra, free.gather(1, (extra.cumsum(1) - 1).clamp(min=0)), parent)
    whole = state["kv_len"].view(b, n)[:, :1].long() // page
    tail = (state["kv_len"].view(b, n)[:, :1] % page).expand(b, n)
    old = table.view(b, n, -1).long()
    entries = torch.arange(old.shape[2], device=old.device)
    row = lambda of: old.gather(1, of[:, :, None].expand(-1, -1, old.shape[2]))  # noqa: E731
    new = torch.where(entries < whole[:, :, None], row(torch.where(valid, parent, place)), row(place))
    copies = extra & valid & (tail > 0)
    at = whole[:, :, None].expand(b, n, 1).clamp(max=old.shape[2] - 1)
    src = torch.where(copies, row(parent.clamp(0, n - 1)).gather(2, at)[..., 0], -1)
    dst = torch.where(copies, row(place).gather(2, at)[..., 0], -1)
    rows = torch.where(copies, tail.long(), 0)
    todo = torch.stack([src, dst, rows], 2).view(b * n, 3)
    real = todo[todo[:, 2] > 0]
    slot = torch.arange(page, device=table.device)[None, None, :, None]
    for name in ("pool_k", "pool_v"):
        for part in _parts(state[name], case):
            if part is not None:
                part[real[:, 1]] = torch.where(slot < real[:, 2, None, None, None], part[real[:, 0]], part[real[:, 1]])
    return new.view(b * n, -1).to(torch.int32), todo.to(torch.int32), state["pool_k"], state["pool_v"]


def _plain_draft(state):
    case, q_start, most = state["case"], state["q_start"], state["most"]
    n = case["new"]
    parent, there = _padded(case, q_start, state["parent"], -1)
    token, _ = _padded(case, q_start, state["token"], -1)
    target, _ = _padded(case, q_start, state["target"], -2)
    above = _ancestors(parent)
    base = state["kv_len"] - q_start[1:] + q_start[:-1]
    pos = (base[:, None] + above.sum(-1) - 1)[there].to(torch.int32)
    mask = _words(above, -(-state["max_new"] // 32))[there]
    # a row agrees when its parent's choice is its token and no earlier sibling's
    rows = torch.arange(n, device=parent.device)
    agrees = there & (parent >= 0) & (parent < rows) & (token == target.gather(1, parent.clamp(min=0).long()))
    earlier = (agrees[:, None, :] & (parent[:, None, :] == parent[:, :, None]) & (rows < rows[:, None])).any(2)
    agrees = (agrees & ~earlier) | ((rows == 0) & there)
    path = there & ~(above & ~agrees[:, None, :]).any(2)
    order = path.cumsum(1) - 1
    path = path & (order < most)
    keep = torch.full((case["batch"], most + 1), -1, dtype=torch.long, device=parent.device)
    keep = keep.scatter(1, torch.where(path, order, most), torch.where(path, rows, -1))[:, :most]
    count = path.sum(1)
    last = torch.where(path, rows, 0).amax(1)
    after = target.gather(1, last[:, None])[:, 0]
    # the kept rows move up to where the cache goes on
    page, at = case["page"], torch.arange(most, device=parent.device)
    moves = keep >= 0
    seq = torch.arange(case["batch"], device=parent.device)[:, None].expand_as(keep)[moves]
    p_from, p_to = (base[:, None] + keep)[moves], (base[:, None] + at).expand_as(keep)[moves]
    table = state["table"].long()
    for name in ("pool_k", "pool_v"):
        for part in _parts(state[name], case):
            if part is not None:
                part[table[seq, p_to // page], :, p_to % page] = part[table[seq, p_from // page], :, p_from % page]
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return pos, mask, i32(keep), i32(count), i32(after), i32(base + count), state["pool_k"], state["pool_v"]


def _plain_tree(state):
    case = state["case"]
    fmt, d, hkv, most = case["fmt"], case["head_dim"], case["kv_heads"], state["table"].shape[1] * case["page"]
    b, new, group = case["batch"], state["max_new"], case["heads"] // hkv
    dev = state["q"].device
    t = torch.arange(state["tokens"], device=dev)
    seq = torch.searchsorted(state["q_start"].long(), t, right=True) - 1
    row = t - state["q_start"].long()[seq]
    table = state["table"].long().clamp(min=0)
    lay = lambda c, s: _values(c[table], None if s is None else s[table], fmt).transpose(1, 2).reshape(b, hkv, most, d)  # noqa: E731
    q = torch.zeros(b, new, case["heads"], d, device=dev)
    q[seq, row] = state["q"] * (1.0 / math.sqrt(d))
    q = q.view(b, new, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * new, d)
    scores = (q @ lay(*_parts(state["pool_k"], case)).transpose(-1, -2)).view(b, hkv, group, new, most)
    base, j = (state["kv_len"] - state["q_start"][1:] + state["q_start"][:-1]).long(), torch.arange(most, device=dev)
    pos = torch.zeros(b, new, dtype=torch.long, device=dev)
    pos[seq, row] = state["pos"].long()
    words = torch.zeros(b, new, state["mask"].shape[1], dtype=torch.int32, device=dev)
    words[seq, row] = state["mask"]
    bits = ((words[..., None] >> torch.arange(32, device=dev)) & 1).flatten(2).bool()  # [b, new, rows]
    ahead = j - base[:, None]  # which of the new tokens a key is
    among = (ahead >= 0) & (j < state["kv_len"][:, None])
    pick = bits.gather(2, ahead.clamp(0, bits.shape[2] - 1)[:, None].expand(b, new, most)) & among[:, None]
    cached = (ahead < 0)[:, None]
    if case["window"]:
        cached = cached & ((j > pos[..., None] - case["window"]) | (j < case["sinks"]))
    scores.masked_fill_(~(cached | pick)[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = (scores.view(b, hkv, group * new, most) @ lay(*_parts(state["pool_v"], case))).view(b, hkv, group, new, d) / total
    return out.permute(0, 3, 1, 2, 4).reshape(b, new, case["heads"], d)[seq, row]


# ---- the definition, in 64 bits ---------------------------------------------
def exact(case, seed):
    s, op, f64 = prepare(case, seed), case["op"], torch.float64
    if op == "rope":
        half, axes = case["rotary"] // 2, case["axes"]
        pos, outs = s["pos"].cpu().numpy().astype(np.float64), []
        angle = np.empty((case["tokens"], half))
        ends = np.cumsum(s["sections"])
        for j in range(half):
            axis = int((ends <= j).sum())
            if case["turns"]:
                axis = j % axes if j < axes * s["sections"][j % axes] else 0
            angle[:, j] = pos[axis] * case["base"] ** (-2.0 * j / case["rotary"])
        turn = torch.polar(torch.ones(angle.shape, dtype=f64), torch.from_numpy(angle)).cuda()[:, None]
        for x in (s["q"], s["k"]):
            y = x.to(f64).clone()
            if case["adjacent"]:
                z = torch.view_as_complex(y[..., : 2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
                y[..., : 2 * half] = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(y[..., :half], y[..., half: 2 * half]) * turn
                y[..., : 2 * half] = torch.cat([z.real, z.imag], -1)
            outs.append(y)
        return tuple(outs)
    if op == "beams":
        n, v, keep = case["beams"], case["vocab"], case["keep"]
        scores, parents, tokens = (np.full((case["groups"], keep), x) for x in (-np.inf, -1.0, -1.0))
        norm = torch.logsumexp(s["logits"].to(f64), 1).cpu().numpy()
        # (of one beam no more than `keep` can be chosen; all at the last one's value or above)
        least = s["logits"].topk(min(keep, v), 1).values[:, -1:]
        rows, cols = (x.cpu().numpy() for x in torch.nonzero(s["logits"] >= least, as_tuple=True))
        x = s["logits"][s["logits"] >= least].to(f64).cpu().numpy()
        before = s["scores"].to(f64).cpu().numpy()
        ended = np.zeros(len(before), dtype=bool) if s["ended"] is None else s["ended"].cpu().numpy() != 0
        live = ~ended[rows]
        score = np.concatenate([(before[rows] + (x - norm[rows]))[live], before[ended]])
        rows = np.concatenate([rows[live], np.nonzero(ended)[0]])
        cols = np.concatenate([cols[live], np.zeros(int(ended.sum()), dtype=cols.dtype)])
        for i in range(case["groups"]):
            here = np.nonzero((rows // n == i) & (score > -np.inf))[0]
            here = here[np.lexsort((cols[here], rows[here], -score[here]))][:keep]
            scores[i, : len(here)], parents[i, : len(here)], tokens[i, : len(here)] = score[here], rows[here] % n, cols[here]
        return torch.from_numpy(scores), torch.from_numpy(parents.astype(np.int32)), torch.from_numpy(tokens.astype(np.int32))
    if op != "tree":
        return None  # whole numbers and bytes
    if work(case)["flops"] > 2e12:
        return None
    news, totals = _lengths(case)
    fmt, d, page = case["fmt"], case["head_dim"], case["page"]

    def kept(pool, i, h):  # the positions of sequence i, head h, from the pool's bytes
        ids, n = s["table"][i, : -(-totals[i] // page)].long(), totals[i]
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

    out = torch.empty(s["tokens"], case["heads"], d, dtype=f64, device="cuda")
    group, at = case["heads"] // case["kv_heads"], 0
    parents = s["parent"].cpu().numpy()
    for i, n in enumerate(news):
        see = np.zeros((n, totals[i]), dtype=bool)
        for r in range(n):
            depth, a = 0, r
            while a >= 0:
                see[r, totals[i] - n + a] = True
                a = parents[at + a]
                depth += 1
            p, j = totals[i] - n + depth - 1, np.arange(totals[i] - n)
            see[r, : totals[i] - n] = (j > p - case["window"]) | (j < case["sinks"]) if case["window"] else True
        hide = torch.from_numpy(~see).cuda()
        for h in range(case["kv_heads"]):
            k, v = kept(s["pool_k"], i, h), kept(s["pool_v"], i, h)
            q = s["q"][at: at + n, h * group: (h + 1) * group].to(f64)
            x = torch.einsum("tgd,kd->gtk", q, k) / math.sqrt(d)
            w = torch.softmax(x.masked_fill(hide, -math.inf), -1)
            out[at: at + n, h * group: (h + 1) * group] = torch.einsum("gtk,kd->tgd", w, v)
        at += n
    return out
