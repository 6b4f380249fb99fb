"""The attention block of a decoder, from prompt to generated tokens.

A fused QKV projection, the paged cache, attention over it and the output
projection with the residual added, all from this library: a batch of prompts
of different lengths goes in as one call (ragged), then every sequence decodes
one token a step, the whole step replayed as a CUDA graph (lengths live on the
device, so the same graph serves every step).

    python examples/attention_block.py [--fmt q8_0] [--cache q8_0] [--batch 8]
        [--prompt 2000] [--steps 64] [--window 0] [--sinks 0]

Prints the time of the prompts and of a decoding step, and checks the last
step against a float32 torch computation from the cache read back
(lq_kv_read).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_gemv_f16w_gb300 as lq  # noqa: E402


class AttentionBlock:
    """Weights, cache and scratch of one layer's attention."""

    def __init__(self, fmt, cache_fmt, embed, heads, kv_heads, head_dim, batch, max_len, page=32, window=0, sinks=0, seed=0):
        self.fmt, self.embed, self.heads, self.kv_heads, self.d = fmt, embed, heads, kv_heads, head_dim
        self.window, self.sinks = window, sinks
        self.wide = (heads + 2 * kv_heads) * head_dim
        gen = torch.Generator().manual_seed(seed)
        pack = lambda n, k: torch.from_numpy(lq.pack(fmt, (torch.randn(n, k, generator=gen) / k**0.5).numpy())).cuda()  # noqa: E731
        self.wqkv, self.wo = pack(self.wide, embed), pack(embed, heads * head_dim)
        pages = -(-max_len // page)
        self.cache = lq.KVCache(cache_fmt, batch * pages, page, kv_heads, head_dim)
        # any assignment of pages to sequences will do; here they alternate
        self.table = torch.arange(batch * pages, dtype=torch.int32).view(pages, batch).t().contiguous().cuda()
        self.work = None

    def __call__(self, x, out, batch):
        """out = x + Wo attention(Wqkv x) for the batch's tokens (rows of x)."""
        n, split = x.shape[0], self.heads * self.d
        qkv = lq.matmul(self.fmt, x, self.wqkv, self.wide, self.embed)
        q, k, v = qkv[:, :split], qkv[:, split:split + self.kv_heads * self.d], qkv[:, split + self.kv_heads * self.d:]
        lq.lq_kv_write(self.cache, batch, k, v)
        if self.work is None:
            self.work = lq.attn_work(self.cache, batch, self.heads)
        o = torch.empty(n, split, device=x.device)
        lq.lq_attn_paged(self.cache, batch, q, o, self.d**-0.5, window=self.window, sinks=self.sinks, work=self.work, heads=self.heads)
        lq.lq_matmul_residual(self.fmt, o, self.wo, x, out, n, self.embed, split)
        return q, o


def attention_in_torch(q, k, v, pos, window, sinks):
    """q [heads, D] at position `pos` over k, v [length, kv_heads, D], float32."""
    j = torch.arange(k.shape[0], device=q.device)
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < sinks)
    group = q.shape[0] // k.shape[1]
    k, v = k[see].repeat_interleave(group, 1), v[see].repeat_interleave(group, 1)
    p = torch.softmax(torch.einsum("hd,jhd->hj", q, k) * q.shape[1]**-0.5, -1)
    return torch.einsum("hj,jhd->hd", p, v)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--fmt", default="q8_0", choices=["f16", "q8_0", "q4_0"], help="weights")
    ap.add_argument("--cache", default="q8_0", choices=["f16", "q8_0", "q4_0"], help="cache")
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=2000, help="the longest prompt")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--embed", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    a = ap.parse_args()
    layer = AttentionBlock(a.fmt, a.cache, a.embed, a.heads, a.kv_heads, a.head_dim, a.batch, a.prompt + a.steps + 8,
                           window=a.window, sinks=a.sinks)

    # prompts of different lengths, one call
    news = [max(1, a.prompt - 37 * i) for i in range(a.batch)]
    tokens = sum(news)
    kv_len = torch.tensor(news, dtype=torch.int32).cuda()
    q_start = torch.cat([torch.zeros(1, dtype=torch.int32), torch.tensor(news).cumsum(0).int()]).cuda()
    x = torch.randn(tokens, a.embed, device="cuda")
    y = torch.empty_like(x)
    prompts = lq.KVBatch(layer.table, kv_len, q_start, tokens, max_q=max(news))
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    layer(x, y, prompts)
    start.record()
    layer(x, y, prompts)
    stop.record()
    torch.cuda.synchronize()
    print(f"{a.batch} prompts, {tokens} tokens: {start.elapsed_time(stop) * 1e3:.0f} us")

    # one token a sequence and step; each step's output is the next one's input
    x = y[(q_start[1:] - 1).long()].clone()
    y = torch.empty_like(x)
    step = lq.KVBatch(layer.table, kv_len, torch.arange(a.batch + 1, dtype=torch.int32).cuda(), a.batch, max_q=1)

    def decode():
        kv_len.add_(1)
        q, o = layer(x, y, step)
        x.copy_(y / y.norm(dim=1, keepdim=True) * a.embed**0.5)
        return q, o

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode()  # once outside the graph
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o = decode()
    start.record()
    for _ in range(a.steps):
        graph.replay()
    stop.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(stop) * 1e3 / a.steps
    print(f"a decoding step of {a.batch} sequences: {us:.1f} us, {a.batch / us * 1e6:.0f} tokens/s and layer")

    # the last step against torch, from what the cache holds
    status = lq.last_device_error()
    if status != lq.LQ_OK:
        raise RuntimeError(f"device status {lq.status_string(status)}")
    worst, lens = 0.0, kv_len.tolist()
    for i, n in enumerate(lens):
        whole = lq.KVBatch(layer.table[i:i + 1].contiguous(), kv_len[i:i + 1], torch.tensor([0, n], dtype=torch.int32).cuda(), n)
        k, v = (torch.empty(n, a.kv_heads, a.head_dim, device="cuda") for _ in range(2))
        lq.lq_kv_read(layer.cache, whole, k, v)
        want = attention_in_torch(q[i].view(a.heads, a.head_dim), k, v, n - 1, a.window, a.sinks)
        worst = max(worst, ((o[i].view_as(want) - want).norm() / want.norm()).item())
    print(f"largest relative difference from torch: {worst:.2g}")
    if not worst < 1e-4:
        raise SystemExit("the last step differs from torch")


if __name__ == "__main__":
    main()
