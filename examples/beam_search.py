"""Beam search over a paged, block-scaled key-value cache, nothing of it on the host.

    python examples/beam_search.py [--fmt mxfp8] [--beams 4] [--steps 40]

A small model of attention layers with NVFP4 projections (heads normed and rotated) and an NVFP4
output layer.  Prompts of different lengths go in packed; then every step is one captured HIP graph: pages
for the new tokens, the layers (norm, rotation and cache write in one call, attention over the cache),
the selection over beams and vocabulary, the block tables of the chosen beams, copies of their partly filled
pages, and the pages that nobody holds any more back on the free list.  Synthetic weights.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp4_04_amd as fp4  # noqa: E402

END = 0  # the token that ends a text


def linear(x, w, w_dec):
    return fp4.gemm_w4a16_decode(x, w_dec) if x.shape[0] <= 16 else fp4.gemm_w4a16(x, w)


class Model:
    def __init__(self, layers, vocab, width, heads, kv_heads, dim, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.freqs = fp4.rope_frequencies(dim)
        self.embedding = normal(vocab, width).to(torch.bfloat16)
        self.layers = []
        for _ in range(layers):
            w_in = fp4.nvfp4_quantize(normal((heads + 2 * kv_heads) * dim, width) * width ** -0.5)
            w_out = fp4.nvfp4_quantize(normal(width, heads * dim) * (heads * dim) ** -0.5)
            norms = [1.0 + 0.1 * normal(dim) for _ in range(2)]
            self.layers.append((w_in, fp4.nvfp4_pack_decode(w_in), w_out, fp4.nvfp4_pack_decode(w_out), *norms))
        # logits of a few units, so that beams compete
        self.head = fp4.nvfp4_quantize(normal(vocab, width) * (3.0 * width ** -0.5))
        self.head_dec = fp4.nvfp4_pack_decode(self.head)

    def projected(self, layer, x):
        """q, k and v as views of one projection's output."""
        w, w_dec = self.layers[layer][:2]
        y = linear(self.normed(x), w, w_dec).view(x.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        return y.split([self.heads, self.kv_heads, self.kv_heads], 1)

    @staticmethod
    def normed(x):
        y = x.float()
        return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def forward(self, tokens, plan, caches, attend):
        x = self.embedding[tokens]
        for i, cache in enumerate(caches):
            q, k, v = self.projected(i, x)
            *_, w_out, w_out_dec, q_norm, k_norm = self.layers[i]
            q = fp4.qk_norm_rope_append(cache, q, k, v, plan.positions, plan.slots, self.freqs, q_norm, k_norm, eps=1e-6)
            x = x + linear(attend(q, cache).reshape(x.shape[0], -1), w_out, w_out_dec)
        return x

    def logits(self, x):
        return linear(self.normed(x), self.head, self.head_dec)


class Search:
    """The state of a batch of beam searches: one row of the block table a beam."""

    def __init__(self, model, fmt, batch, beams, most, page, layers):
        self.model, self.batch, self.beams, self.page = model, batch, beams, page
        rows, width = batch * beams, (most + page - 1) // page
        pages = rows * width + 1
        ts = [None, None]
        if fmt == "nvfp4":  # second-level scales with headroom for normed keys and projected values
            ts = [torch.full((model.kv_heads,), 8.0 / 2688, device="cuda") for _ in range(2)]
        self.caches = [fp4.KVCache.alloc(fmt, pages, model.kv_heads, page, model.dim, "cuda", *ts) for _ in range(layers)]
        self.pool = fp4.KVPages.alloc(pages, page)
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.scores = torch.zeros(batch, beams, device="cuda")
        self.done = torch.zeros(batch, beams, dtype=torch.bool, device="cuda")
        self.tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.parents = torch.zeros(batch, beams, dtype=torch.int32, device="cuda")
        self.one = torch.ones(rows, dtype=torch.int32, device="cuda")

    def start(self, prompts):
        """The prompts go into the first row of each group, the other rows come to share its pages."""
        model, batch, beams, page = self.model, self.batch, self.beams, self.page
        counts = torch.tensor([len(p) for p in prompts], dtype=torch.int32)
        new = torch.zeros(batch, beams, dtype=torch.int32)
        new[:, 0] = counts
        total = int(counts.sum())
        plan = fp4.kv_pages_extend(self.pool, self.table, self.lens, new.view(-1).cuda(), total)

        def attend(q, cache):
            k, v = fp4.kv_cache_read(cache, self.table, plan.cu_k, total)
            return fp4.attn_prefill(q, k, v, plan.cu_q, plan.cu_k)

        x = model.forward(torch.tensor(sum(prompts, []), device="cuda"), plan, self.caches, attend)
        last = x[counts.cumsum(0).cuda() - 1]

        # Full pages are shared.  The other rows ask for a page for the prompt's tail, and get it copied
        # as children of the first.
        table, lens = self.table.view(batch, beams, -1), self.lens.view(batch, beams)
        table[:, 1:] = table[:, :1]
        tail = lens[:, :1] % page
        lens[:, 1:] = lens[:, :1] - tail
        new = tail.expand(batch, beams).clone()
        new[:, 0] = 0
        fp4.kv_pages_extend(self.pool, self.table, self.lens, new.view(-1), batch * beams * page)
        self.reorder(torch.zeros(batch, beams, dtype=torch.int32, device="cuda"))
        # the first tokens: of each group's one row, as many continuations as there are beams
        self.scores, self.first_parents, tokens = fp4.beam_select(model.logits(last), torch.zeros(batch, 1, device="cuda"), k=beams)
        self.tokens.copy_(tokens.view(-1))
        self.done = tokens == END

    def reorder(self, parents):
        copies = fp4.kv_pages_reorder(self.table, self.lens, parents, self.page)
        for cache in self.caches:
            fp4.kv_cache_copy(cache, copies)

    def step(self):
        """The last selection's tokens go in, the next ones are selected."""
        plan = fp4.kv_pages_extend(self.pool, self.table, self.lens, self.one, self.one.shape[0], offsets=False)
        x = self.model.forward(self.tokens, plan, self.caches,
                               lambda q, cache: fp4.attn_decode_paged(q, cache, self.table, self.lens))
        scores, parents, tokens = fp4.beam_select(self.model.logits(x), self.scores, done=self.done, end_token=END)
        self.reorder(parents)
        fp4.kv_pages_collect(self.pool, self.table, self.lens)
        done = self.done.gather(1, parents.long()) | (tokens == END)
        self.scores.copy_(scores)
        self.parents.copy_(parents)
        self.tokens.copy_(tokens.view(-1))
        self.done.copy_(done)


def run(fmt="mxfp8", prompts=(37, 5, 64), beams=4, steps=20, layers=2, vocab=1000, width=512, heads=8, kv_heads=2, dim=64,
        page=16, seed=0, graph=True):
    """(texts, scores, search): of every group its beams' tokens (prompt included; the last one is not in the cache yet),
    best first."""
    model = Model(layers, vocab, width, heads, kv_heads, dim, seed)
    g = torch.Generator().manual_seed(seed + 1)
    prompts = [torch.randint(1, vocab, (n,), generator=g).tolist() for n in prompts]
    search = Search(model, fmt, len(prompts), beams, max(map(len, prompts)) + steps, page, layers)
    search.start(prompts)
    texts = [[p + [int(t)] for t in row] for p, row in zip(prompts, search.tokens.view(-1, beams))]

    step = search.step
    if graph:
        # The warm-up changes the state, which is put back.  The pages may stay as they are: here all beams of a group
        # still hold the same text, and the slots behind it are written again.
        kept = [t.clone() for t in (search.table, search.lens, search.pool.free, search.pool.state, search.scores, search.tokens, search.done)]
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        for t, old in zip((search.table, search.lens, search.pool.free, search.pool.state, search.scores, search.tokens, search.done), kept):
            t.copy_(old)
        step = captured.replay
    for _ in range(steps - 1):
        step()
        tokens, parents = search.tokens.view(-1, beams).tolist(), search.parents.tolist()
        texts = [[rows[p] + [t] for p, t in zip(ps, ts)] for rows, ps, ts in zip(texts, parents, tokens)]
    return texts, search.scores, search


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--fmt", choices=["bf16", "mxfp8", "nvfp4", "mxfp4"], default=None, help="cache format (default: all)")
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    for fmt in [a.fmt] if a.fmt else ["bf16", "mxfp8", "nvfp4", "mxfp4"]:
        texts, scores, search = run(fmt, beams=a.beams, steps=a.steps)
        free, refused = search.pool.state.tolist()
        print(f"{fmt:6s} best scores {[round(float(s), 3) for s in scores[:, 0]]}, {search.pool.pages - free} of "
              f"{search.pool.pages} pages held for {len(texts) * a.beams} beams, {refused} requests refused")


if __name__ == "__main__":
    main()
