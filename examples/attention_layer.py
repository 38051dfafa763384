"""One attention layer served with block-scaled weights and a block-scaled key-value cache.

    python examples/attention_layer.py [--fmt mxfp8] [--steps 64]

The layer's q/k/v and output projections are NVFP4 weights (W4A16 GEMMs: the row-major form
for prompts, the decode layout for single tokens).  Prompts of different lengths arrive
packed, in two chunks each: a chunk's keys and values are quantized into the paged cache, the
contexts are read back, and the chunk attends to them.  Then every sequence generates: one
captured HIP graph per step appends the new token and attends over the cache.  Synthetic
weights and inputs; every step's output is compared with a plain fp32 layer that keeps its
keys and values as they are, so the difference shows what the cache format costs.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp4_04_amd as fp4  # noqa: E402


class AttentionLayer:
    def __init__(self, width, heads, kv_heads, dim, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        w_in = torch.randn((heads + 2 * kv_heads) * dim, width, device="cuda", generator=g) * width ** -0.5
        w_out = torch.randn(width, heads * dim, device="cuda", generator=g) * (heads * dim) ** -0.5
        self.w_in, self.w_out = fp4.nvfp4_quantize(w_in), fp4.nvfp4_quantize(w_out)
        self.w_in_dec, self.w_out_dec = fp4.nvfp4_pack_decode(self.w_in), fp4.nvfp4_pack_decode(self.w_out)

    def project(self, x):
        """x [tokens, width] -> q, k, v as views of one projection's output."""
        y = fp4.gemm_w4a16_decode(x, self.w_in_dec) if x.shape[0] <= 16 else fp4.gemm_w4a16(x, self.w_in)
        y = y.view(x.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        return y.split([self.heads, self.kv_heads, self.kv_heads], 1)

    def output(self, o):
        o = o.reshape(o.shape[0], -1)
        return fp4.gemm_w4a16_decode(o, self.w_out_dec) if o.shape[0] <= 16 else fp4.gemm_w4a16(o, self.w_out)


class Pages:
    """Pages of a cache, dealt to sequences as they grow (host side)."""

    def __init__(self, cache, seqs, most):
        self.page = cache.page_size
        self.table = torch.full((seqs, (most + self.page - 1) // self.page), -1, dtype=torch.int32)
        self.free = torch.randperm(cache.pages).tolist()
        self.lens = [0] * seqs

    def grow(self, by):
        """`by` new tokens of every sequence: their slots."""
        slots = []
        for b, n in enumerate(by):
            for pos in range(self.lens[b], self.lens[b] + n):
                if pos % self.page == 0:
                    self.table[b, pos // self.page] = self.free.pop()
                slots.append(int(self.table[b, pos // self.page]) * self.page + pos % self.page)
            self.lens[b] += n
        return torch.tensor(slots, dtype=torch.int64, device="cuda")


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def plain_attention(q, k, v, scale):
    """The last q.shape[0] positions of one sequence in fp32: q [n, heads, dim], k, v [keys, kv heads, dim]."""
    n, keys, group = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    k, v = (x.float().repeat_interleave(group, 1).transpose(0, 1).contiguous() for x in (k, v))
    z = torch.matmul(q.float().transpose(0, 1), k.transpose(1, 2).contiguous()) * scale
    at = torch.arange(keys, device=q.device)
    z.masked_fill_(at > (keys - n + torch.arange(n, device=q.device))[:, None], float("-inf"))
    return torch.matmul(torch.softmax(z, -1), v).transpose(0, 1)


def run(fmt="mxfp8", prompts=(700, 33, 1, 260), steps=16, width=1024, heads=16, kv_heads=4, dim=64, page=32, seed=0):
    layer = AttentionLayer(width, heads, kv_heads, dim, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    seqs, most = len(prompts), max(prompts) + steps
    ts = [None, None]
    if fmt == "nvfp4":  # second-level scales from the range of a normal projection, with headroom
        ts = [torch.full((kv_heads,), 8.0 / 2688, device="cuda") for _ in range(2)]
    cache = fp4.KVCache.alloc(fmt, sum((p + steps + page - 1) // page for p in prompts), kv_heads, page, dim, "cuda", *ts)
    pages, scale = Pages(cache, seqs, most), dim ** -0.5
    kept = [([], []) for _ in prompts]  # the plain layer's keys and values
    worst = 0.0

    def compare(o, q, ks, vs, counts):
        nonlocal worst
        at = 0
        for b, n in enumerate(counts):
            if n == 0:
                continue
            kept[b][0].append(ks[at:at + n].clone())
            kept[b][1].append(vs[at:at + n].clone())
            want = plain_attention(q[at:at + n], torch.cat(kept[b][0]), torch.cat(kept[b][1]), scale)
            got = o[at:at + n].float()
            worst = max(worst, float((got - want).norm() / want.norm()))
            at += n

    # ---- prompts, in two chunks
    for counts in ([p // 2 for p in prompts], [p - p // 2 for p in prompts]):
        x = torch.randn(sum(counts), width, device="cuda", generator=g).to(torch.bfloat16)
        q, k, v = layer.project(x)
        fp4.kv_cache_append(cache, k, v, pages.grow(counts))
        table, whole = pages.table.cuda(), sum(pages.lens)
        kc, vc = fp4.kv_cache_read(cache, table, offsets(pages.lens), whole)
        o = fp4.attn_prefill(q, kc, vc, offsets(counts), offsets(pages.lens))
        y = layer.output(o)
        compare(o, q, k, v, counts)

    # ---- one token of every sequence at a time, the step captured once
    x = torch.zeros(seqs, width, dtype=torch.bfloat16, device="cuda")
    slots = torch.full((seqs,), -1, dtype=torch.int64, device="cuda")  # the warm-up stores nothing
    table = pages.table.cuda()
    lens = torch.tensor(pages.lens, dtype=torch.int32, device="cuda")
    space = fp4.attn_decode_paged_workspace(cache, seqs, heads, table.shape[1])

    def step():
        q, k, v = layer.project(x)
        fp4.kv_cache_append(cache, k, v, slots)
        o = fp4.attn_decode_paged(q, cache, table, lens, workspace=space)
        return q, k, v, o, layer.output(o)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, k, v, o, y = step()
    for _ in range(steps):
        x.copy_(torch.randn(seqs, width, device="cuda", generator=g))
        slots.copy_(pages.grow([1] * seqs))
        table.copy_(pages.table)
        lens.copy_(torch.tensor(pages.lens, dtype=torch.int32))
        graph.replay()
        compare(o, q, k, v, [1] * seqs)
    return worst, cache.nbytes(), y


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--fmt", choices=["bf16", "mxfp8", "nvfp4", "mxfp4"], default=None, help="cache format (default: all)")
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    for fmt in [a.fmt] if a.fmt else ["bf16", "mxfp8", "nvfp4", "mxfp4"]:
        worst, nbytes, _ = run(fmt, steps=a.steps)
        print(f"{fmt:6s} cache {nbytes / 1e6:6.2f} MB, largest relative error of a sequence's attention output {worst:.4f}")


if __name__ == "__main__":
    main()
