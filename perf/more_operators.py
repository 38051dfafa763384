"""What surrounds attention in a generate loop over the paged cache: what is measured.

Six calls of a serving step, each in a plain form (elementary torch operations) and as the
library's own:

* ``rotate``: queries and keys of every head are normed and rotated by their positions.
* ``store``: the same, with the keys and the values quantized into the paged cache.
* ``extend``: pages for new tokens are dealt to sequences; slots, positions and offsets follow.
* ``collect``: pages that no sequence holds any more go back to the free list.
* ``select``: the best continuations of every group of beams over the whole vocabulary.
* ``reorder``: the beams' block tables follow the selection, partly filled pages are copied.

A slot is page * page_size + offset; a sequence's pages stand in its row of the block table,
unused entries of which are -1.  Cache tensors: codes [pages, heads, page, row], scale bytes
[pages, heads, head_dim / 32, page].
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one chat user's new token in one layer: latency
        {"name": "rotate_one", "op": "rotate", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "norm": True, "by_head": False, "dtype": "bf16", "far": 4096},
        # a few prompts of a small model: odd head size, part of it rotated in neighbouring pairs, fp32, no norm
        {"name": "rotate_odd_fp32", "op": "rotate", "tokens": 1537, "heads": 10, "kv_heads": 10, "dim": 80, "rot": 32,
         "interleaved": True, "norm": False, "by_head": False, "dtype": "fp32", "far": 1 << 20},
        # prompts of a whole batch; heads of a 5120-wide layer, positions of a long context
        {"name": "rotate_prompt", "op": "rotate", "tokens": 16384, "heads": 40, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "norm": True, "by_head": True, "dtype": "bf16", "far": 131072},
        # one decode step of a serving batch: new keys and values go into an MXFP8 cache
        {"name": "store_step_mxfp8", "op": "store", "fmt": "mxfp8", "tokens": 64, "heads": 40, "kv_heads": 8,
         "dim": 128, "rot": 128, "interleaved": False, "norm": True, "by_head": False, "page": 64, "far": 16384},
        # a chunk of prompts into a bf16 cache, wide heads of which a quarter turns
        {"name": "store_chunk_bf16", "op": "store", "fmt": "bf16", "tokens": 6001, "heads": 16, "kv_heads": 4,
         "dim": 256, "rot": 64, "interleaved": False, "norm": True, "by_head": False, "page": 32, "far": 8192},
        # one decode step of a serving batch: one token each
        {"name": "extend_step", "op": "extend", "seqs": 64, "held": 16384, "new": 1, "page": 64, "short": False},
        # ragged chunks of many prompts, more than the free pages can take
        {"name": "extend_prompts_short", "op": "extend", "seqs": 300, "held": 3000, "new": 900, "page": 16,
         "short": True},
        # a large pool after many sequences ended
        {"name": "collect_pool", "op": "collect", "seqs": 512, "held": 8192, "page": 16, "ended": 0.3},
        # one user's four beams
        {"name": "select_one", "op": "select", "batch": 1, "beams": 4, "vocab": 32000, "k": 4, "dtype": "bf16",
         "ended": 0.0},
        # beams of a serving batch over a large vocabulary, twice as many candidates as beams, some beams ended
        {"name": "select_batch", "op": "select", "batch": 64, "beams": 8, "vocab": 131072, "k": 16, "dtype": "bf16",
         "ended": 0.1},
        # one user's four beams, short prompt
        {"name": "reorder_one", "op": "reorder", "fmt": "bf16", "batch": 1, "beams": 4, "prompt": 333, "made": 77,
         "kv_heads": 8, "dim": 128, "page": 16},
        # a batch of beams after a few hundred tokens
        {"name": "reorder_batch_mxfp8", "op": "reorder", "fmt": "mxfp8", "batch": 48, "beams": 6, "prompt": 1000,
         "made": 500, "kv_heads": 4, "dim": 128, "page": 64},
    ]


def _log(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "store", "extend", "collect", "select", "select", "reorder"])
    kv = rng.choice([1, 2, 3, 4, 5, 8, 12])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    while kv * group > 40:
        group = max(1, group // 2)
    if op in ("rotate", "store"):
        dim = rng.choice([64, 128, 128, 256] if op == "store" else [48, 64, 80, 96, 128, 128, 160, 192, 256])
        rot = rng.choice([dim, dim, dim // 2 // 16 * 16, min(dim, 32)])
        case = {"op": op, "heads": kv * group, "kv_heads": kv, "dim": dim, "rot": rot,
                "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.8, "by_head": rng.random() < 0.3,
                "far": _log(rng, 16, 1 << 20)}
        case["tokens"] = _log(rng, 1, int(16384 * 48 * 128 / ((kv * group + 2 * kv) * dim) / 2))
        if op == "rotate":
            case["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        else:
            case["fmt"], case["page"] = rng.choice(["bf16", "mxfp8"]), rng.choice([16, 32, 64, 128])
        return case
    if op in ("extend", "collect"):
        case = {"op": op, "seqs": _log(rng, 1, 1024), "page": rng.choice([16, 32, 64, 128])}
        case["held"] = _log(rng, 1, min(131072, 4194304 // case["seqs"]))
        if op == "collect":
            case["ended"] = rng.choice([0.0, 0.1, 0.5, 1.0])
        else:
            case["new"] = rng.choice([1, _log(rng, 1, min(32768, 262144 // case["seqs"]))])
            case["short"] = rng.random() < 0.3
        return case
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        case = {"op": op, "beams": beams, "batch": _log(rng, 1, max(1, 256 // beams)), "vocab": _log(rng, 200, 262144),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "ended": rng.choice([0.0, 0.0, 0.2])}
        while beams * case["batch"] * case["vocab"] > 512 * 131072 // 2:
            case["vocab"] //= 2
        case["k"] = rng.choice([beams, 2 * beams])
        return case
    beams = rng.choice([2, 3, 4, 5, 8, 16])
    case = {"op": op, "fmt": rng.choice(["bf16", "mxfp8"]), "beams": beams, "batch": _log(rng, 1, 256 // beams),
            "prompt": _log(rng, 1, 2000), "made": _log(rng, 1, 600), "kv_heads": rng.choice([1, 2, 4, 8]),
            "dim": rng.choice([64, 128, 128, 256]), "page": rng.choice([16, 32, 64])}

    def size():
        tokens = case["batch"] * (case["prompt"] + beams * (case["made"] + case["page"]))
        return tokens * case["kv_heads"] * case["dim"] * (2 if case["fmt"] == "bf16" else 1)

    while size() > 150e6 and case["batch"] > 1:
        case["batch"] //= 2
    while size() > 150e6:
        case["made"], case["prompt"] = case["made"] // 2 + 1, case["prompt"] // 2 + 1
    return case


def _counts(case):
    """extend, collect: tokens held and new of each sequence, spread over the logarithm, some of them 0; of
    one-token steps (new == 1) every sequence takes one."""
    rng = random.Random(case["seqs"] * 1000003 + case["held"])
    held = [0 if rng.random() < 0.05 else _log(rng, 1, case["held"]) for _ in range(case["seqs"])]
    if case["op"] == "collect":
        return [0 if rng.random() < case["ended"] else n for n in held], held
    new = [1 if case["new"] == 1 else 0 if rng.random() < 0.05 else _log(rng, 1, case["new"]) for _ in held]
    return held, new


def _pages(n, page):
    return (n + page - 1) // page


def work(case):
    op = case["op"]
    if op in ("rotate", "store"):
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        if op == "rotate":
            return {"bytes": values * 2.0 * (2 if case["dtype"] == "bf16" else 4) + 4.0 * case["tokens"],
                    "flops": 10.0 * values}
        stored = 2 * case["tokens"] * case["kv_heads"] * case["dim"]
        q = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": q * 4.0 + stored * (2 + (2 if case["fmt"] == "bf16" else 33 / 32)) + 12.0 * case["tokens"],
                "flops": 10.0 * values + 4.0 * stored}
    if op in ("extend", "collect"):
        first, second = _counts(case)
        if op == "collect":
            live = sum(_pages(n, case["page"]) for n in first)
            total = sum(_pages(n, case["page"]) for n in second) + case["seqs"]
            return {"bytes": 4.0 * (live + case["seqs"] + total - live), "flops": 1.0 * (live + total)}
        made = sum(_pages(a + b, case["page"]) - _pages(a, case["page"]) for a, b in zip(first, second))
        tokens = sum(second)
        return {"bytes": 12.0 * tokens + 8.0 * made + 20.0 * case["seqs"], "flops": 4.0 * tokens}
    if op == "select":
        values = case["batch"] * case["beams"] * case["vocab"] * (1.0 - case["ended"])
        return {"bytes": values * (2 if case["dtype"] == "bf16" else 4) + 12.0 * case["batch"] * (case["beams"] + case["k"]),
                "flops": 4.0 * values}
    rows, n = case["batch"] * case["beams"], case["prompt"] + case["made"]
    # of `beams` draws with replacement about (1 - 1/beams)^beams leave a row without a child
    copied = rows * (1.0 - 1.0 / case["beams"]) ** case["beams"] * (n % case["page"])
    token = 2 * case["kv_heads"] * case["dim"] * (2 if case["fmt"] == "bf16" else 33 / 32)
    return {"bytes": 8.0 * rows * _pages(n, case["page"]) + 2.0 * copied * token + 20.0 * rows,
            "flops": 1.0 * rows * _pages(n, case["page"])}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _projected(g, tokens, heads, dim, dtype):
    """q, k and v of one projection: columns of its rows, a few channels much larger than the others."""
    x = torch.randn(tokens, heads, dim, device="cuda", generator=g)
    gain = torch.ones(heads, dim, device="cuda")
    gain[torch.rand(heads, dim, device="cuda", generator=g) < 0.03] = 6.0
    return (x * gain).to(dtype)


def _table(rows, pages, seed):
    """Rows of page counts -> a block table over `pages` pages in random order, and the pages left over."""
    width = max(1, max(rows))
    used = torch.arange(width).unsqueeze(0) < torch.tensor(rows).unsqueeze(1)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(rows), width), -1, dtype=torch.int32)
    table[used] = order[:sum(rows)]
    return table, order[sum(rows):]


def _empty_cache(fmt, pages, kv_heads, page, dim, g):
    """Some contents: what an earlier use of the pages has left there."""
    shape = (pages, kv_heads, page, dim)
    if fmt == "bf16":
        c = {s + "_codes": torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16) for s in "kv"}
        return {"fmt": fmt, **c, "k_scales": None, "v_scales": None}
    c = {s + "_codes": torch.randint(0, 120, shape, device="cuda", generator=g, dtype=torch.uint8) for s in "kv"}
    for s in "kv":
        c[s + "_scales"] = torch.randint(118, 121, (pages, kv_heads, dim // 32, page), device="cuda", generator=g,
                                         dtype=torch.uint8)
    return {"fmt": fmt, **c}


def _prepare_heads(case, g, seed):
    heads, kv, dim, n = case["heads"], case["kv_heads"], case["dim"], case["tokens"]
    dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    whole = _projected(g, n, heads + 2 * kv, dim, dtype)
    s = {"q": whole[:, :heads], "k": whole[:, heads:heads + kv], "v": whole[:, heads + kv:]}
    s["positions"] = torch.randint(0, case["far"], (n,), device="cuda", generator=g, dtype=torch.int32)
    at = torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda")
    s["freqs"] = 10000.0 ** (-at / case["rot"]) if case["rot"] else None
    s["q_weight"] = s["k_weight"] = s["eps"] = None
    if case["norm"]:
        s["eps"] = 1e-6
        for x, h in (("q", heads), ("k", kv)):
            shape = (h, dim) if case["by_head"] else (dim,)
            s[x + "_weight"] = 1.0 + 0.2 * torch.randn(shape, device="cuda", generator=g)
    if case["op"] == "store":
        page = case["page"]
        pages = _pages(n, page) + 7
        s["cache"] = _empty_cache(case["fmt"], pages, kv, page, dim, g)
        # consecutive tokens mostly stand in one page; every 50th is padding
        order = torch.randperm(pages, device="cuda", generator=g)
        t = torch.arange(n, device="cuda")
        s["slots"] = order[t // page] * page + t % page
        s["slots"][t % 50 == 49] = -1
    return s


def _prepare_pages(case, g, seed):
    first, second = _counts(case)
    page = case["page"]
    s = {}
    if case["op"] == "collect":
        table, left = _table([_pages(n, page) for n in second], sum(_pages(n, page) for n in second) + case["seqs"], seed)
        s["seq_lens"] = torch.tensor(first, dtype=torch.int32)
    else:
        after = [_pages(a + b, page) for a, b in zip(first, second)]
        held = [_pages(a, page) for a in first]
        need = sum(after) - sum(held)
        count = int(need * 0.7) if case["short"] else need + 5
        table, left = _table(held, sum(held) + count + 3, seed)
        wide = torch.full((case["seqs"], max(1, max(after))), -1, dtype=torch.int32)
        wide[:, :table.shape[1]] = table[:, :wide.shape[1]]
        table, left = wide, left[:count]
        s["seq_lens"] = torch.tensor(first, dtype=torch.int32).cuda()
        s["new_lens"] = torch.tensor(second, dtype=torch.int32).cuda()
        s["tokens"] = sum(second)
    s["pages"] = sum(_pages(n, page) for n in second) + case["seqs"] if case["op"] == "collect" else sum(held) + count + 3
    s["free"] = torch.full((s["pages"],), -1, dtype=torch.int32)
    s["free"][:len(left)] = left
    s["state"] = torch.tensor([len(left), 0], dtype=torch.int32).cuda()
    for x in ("seq_lens", "free"):
        s[x] = s[x].cuda()
    s["table"] = table.cuda()
    return s


def _prepare_select(case, g, seed):
    rows, vocab = case["batch"] * case["beams"], case["vocab"]
    x = 2.0 * torch.randn(rows, vocab, device="cuda", generator=g)
    # some tokens that the context makes likely, partly the same ones in every beam
    few = max(1, min(vocab // 8, 40))
    at = torch.randint(0, vocab, (rows, few), device="cuda", generator=g)
    x.scatter_add_(1, at, 6.0 * torch.rand(rows, few, device="cuda", generator=g))
    s = {"logits": x.to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)}
    s["scores"] = -20.0 * torch.rand(case["batch"], case["beams"], device="cuda", generator=g)
    s["done"] = None
    if case["ended"]:
        s["done"] = torch.rand(case["batch"], case["beams"], device="cuda", generator=g) < case["ended"]
    return s


def _prepare_reorder(case, g, seed):
    batch, beams, page = case["batch"], case["beams"], case["page"]
    n = case["prompt"] + case["made"]
    shared, width = case["prompt"] // page, _pages(n, page)
    mine = width - shared
    pages = batch * (shared + beams * mine) + 3
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((batch, beams, width + 4), -1, dtype=torch.int32, device="cuda")
    table[:, :, :shared] = order[:batch * shared].view(batch, 1, shared)
    table[:, :, shared:width] = order[batch * shared:batch * (shared + beams * mine)].view(batch, beams, mine)
    s = {"table": table.view(batch * beams, -1), "pages": pages}
    s["seq_lens"] = torch.full((batch * beams,), n, dtype=torch.int32, device="cuda")
    s["parents"] = torch.randint(0, beams, (batch, beams), device="cuda", generator=g, dtype=torch.int32)
    s["cache"] = _empty_cache(case["fmt"], pages, case["kv_heads"], page, case["dim"], g)
    s["table_out"] = torch.full_like(s["table"], -1)  # the step's other table
    return s


def prepare(case, seed):
    make = {"rotate": _prepare_heads, "store": _prepare_heads, "extend": _prepare_pages, "collect": _prepare_pages,
            "select": _prepare_select, "reorder": _prepare_reorder}
    s = make[case["op"]](case, _gen(seed), seed)
    s["case"] = case
    if own:
        import block_scaled_fp4_04_amd as fp4

        s["fp4"] = fp4
        if "cache" in s:  # the handles that a program keeps
            s["handle"] = fp4.KVCache(**s["cache"])
        if "free" in s:
            s["pool"] = fp4.KVPages(s["free"], s["state"], case["page"])
    return s


# ------------------------------------------------------------- plain form --

def _turned(x, positions, freqs, rot, interleaved):
    """The first `rot` values of rows x [tokens, heads, dim] turned by positions * freqs."""
    if rot == 0:
        return x
    a = positions.double()[:, None] * freqs
    c, s = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    y = x[..., :rot]
    if interleaved:
        u, w = y[..., 0::2], y[..., 1::2]
        y = torch.stack([u * c - w * s, w * c + u * s], -1).flatten(-2)
    else:
        u, w = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([u * c - w * s, w * c + u * s], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _rows(s, x):
    case, y = s["case"], s[x].float()
    if s["eps"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * s[x + "_weight"]
    return _turned(y, s["positions"], s["freqs"], case["rot"], case["interleaved"])


def _held(c):
    """What the cache holds: its values' and scales' types say what they stand for."""
    if c["fmt"] == "bf16":
        return {"k": c["k_codes"], "v": c["v_codes"]}
    return {"k": c["k_codes"].view(torch.float8_e4m3fn), "v": c["v_codes"].view(torch.float8_e4m3fn),
            "k_scales": c["k_scales"].view(torch.float8_e8m0fnu), "v_scales": c["v_scales"].view(torch.float8_e8m0fnu)}


def _plain_rotate(s):
    dtype = s["q"].dtype
    return {"q": _rows(s, "q").to(dtype), "k": _rows(s, "k").to(dtype)}


def _plain_put(c, x, rows, slots):
    kept = slots >= 0
    rows, slots = rows[kept], slots[kept]
    page = c[x + "_codes"].shape[2]
    at, off = slots // page, slots % page
    if c["fmt"] == "bf16":
        c[x + "_codes"][at, :, off] = rows.to(torch.bfloat16)
        return
    b = rows.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    # the power of two that takes the block's largest value to the top binade of E4M3
    e = torch.where(amax > 0, (torch.frexp(amax).exponent - 9).clamp(-127, 127), -127)
    codes = torch.ldexp(b, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    c[x + "_codes"][at, :, off] = codes
    c[x + "_scales"].transpose(2, 3)[at, :, off] = (e + 127).to(torch.uint8).squeeze(-1)


def _plain_store(s):
    _plain_put(s["cache"], "k", _rows(s, "k"), s["slots"])
    _plain_put(s["cache"], "v", s["v"].float(), s["slots"])
    return {"q": _rows(s, "q").to(torch.bfloat16), **_held(s["cache"])}


def _plain_extend(s):
    page, tokens, table = s["case"]["page"], s["tokens"], s["table"]
    old, n, count = s["seq_lens"].long(), s["new_lens"].long(), s["state"][0].long()
    width, seqs = table.shape[1], table.shape[0]
    cum = n.cumsum(0)
    fits = (old + n <= width * page) & (cum <= tokens)
    have = (old + page - 1) // page
    need = torch.where(fits, (old + n + page - 1) // page - have, 0)
    before = need.cumsum(0)
    given = fits & ((need == 0) | (before <= count))
    lens = torch.where(given, old + n, old)
    taken = torch.where(given & (need > 0), before, 0).amax()
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cum, t, right=True).clamp(max=seqs - 1)
    pos = old[b] + t - (cum - n)[b]
    at = pos // page
    fresh = at - have[b]
    place = (count - 1 - (before - need)[b] - fresh).clamp(0, s["pages"] - 1)
    ids = torch.where(fresh >= 0, s["free"].long()[place], table[b, at.clamp(max=width - 1)].long())
    slots = torch.where(given[b], ids * page + pos % page, -1)
    # the tokens that begin a page write its table entry
    flat = torch.cat([table.flatten(), table.new_zeros(1)])
    flat[torch.where(given[b] & (pos % page == 0), b * width + at, seqs * width)] = ids.to(torch.int32)
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    return {"slots": slots, "positions": pos.to(torch.int32), "cu_q": torch.cat([zero, cum]).to(torch.int32),
            "cu_k": torch.cat([zero, lens.cumsum(0)]).to(torch.int32), "seq_lens": lens.to(torch.int32),
            "table": flat[:-1].view(seqs, width),
            "state": torch.stack([count - taken, (~given & (n > 0)).sum() + s["state"][1]]).to(torch.int32)}


def _plain_collect(s):
    page, pages, table = s["case"]["page"], s["pages"], s["table"]
    live = torch.arange(table.shape[1], device="cuda") < ((s["seq_lens"] + page - 1) // page)[:, None]
    used = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
    used[torch.where(live, table, pages).flatten().long()] = True
    free = ~used[:pages]
    rank = free.long().cumsum(0) - 1
    out = torch.cat([s["free"], s["free"].new_zeros(1)])
    out[torch.where(free, rank, pages)] = torch.arange(pages, dtype=torch.int32, device="cuda")
    return {"free": out[:-1], "count": free.sum().to(torch.int32).view(1)}


END = 2  # the token that ends a text


def _best(total, scores, done, k):
    """The k best of total [batch, beams, vocab] in 64 bits, ties to the lowest place."""
    batch, beams, vocab = total.shape
    if done is not None:
        ended = torch.full((vocab,), -math.inf, dtype=torch.float64, device="cuda")
        ended[END] = 0.0
        total = torch.where(done[..., None], scores.double()[..., None] + ended, total)
    total = torch.nan_to_num(total, nan=-math.inf).flatten(1)
    best, at = torch.sort(total, dim=-1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    real = best > -math.inf
    filler = torch.arange(k, device="cuda").clamp(max=beams - 1)
    return {"scores": best.float(), "parents": torch.where(real, at // vocab, filler).to(torch.int32),
            "tokens": torch.where(real, at % vocab, -1).to(torch.int32)}


def _plain_select(s):
    case = s["case"]
    z = s["logits"].double().view(case["batch"], case["beams"], -1)
    total = s["scores"].double()[..., None] + (z - torch.logsumexp(z, -1, keepdim=True))
    return _best(total, s["scores"], s["done"], case["k"])


def _plain_reorder(s):
    case, p = s["case"], s["parents"].long()
    batch, beams, page = case["batch"], case["beams"], case["page"]
    table, out = s["table"].view(batch, beams, -1), s["table_out"].view(batch, beams, -1)
    n = s["seq_lens"].view(batch, beams).long().gather(1, p)
    live = torch.arange(table.shape[2], device="cuda") < ((n + page - 1) // page)[..., None]
    new = torch.where(live, table.gather(1, p[..., None].expand(-1, -1, table.shape[2])), out)
    row = torch.arange(beams, device="cuda")
    further = ((p[:, :, None] == p[:, None, :]) & (row[None, None, :] < row[None, :, None])).any(-1)
    dropped = ~(p[:, :, None] == row).any(1)
    # the m-th further child takes the page of the m-th dropped row
    order = torch.sort((~dropped).int(), dim=-1, stable=True).indices
    heir = order.gather(1, (further.long().cumsum(1) - 1).clamp(min=0))
    at, off = n // page, n % page
    copied = further & (off > 0)
    place = at.clamp(max=table.shape[2] - 1)
    src = table[torch.arange(batch, device="cuda")[:, None], p, place]
    dst = table[torch.arange(batch, device="cuda")[:, None], heir, place]
    new.scatter_(2, place[..., None], torch.where(copied, dst, new.gather(2, place[..., None]).squeeze(2))[..., None])
    copies = torch.stack([torch.where(copied, src, -1), torch.where(copied, dst, -1),
                          torch.where(copied, off, 0).to(torch.int32)], -1).view(-1, 3)
    s["table_out"].copy_(new.view_as(s["table_out"]))
    real = copies[copies[:, 0] >= 0].long()
    src, dst, off = real[:, 0], real[:, 1], real[:, 2]
    kept = torch.arange(page, device="cuda") < off[:, None]
    c = s["cache"]
    for x in ("k", "v"):
        codes, scales = c[x + "_codes"], c[x + "_scales"]
        codes[dst] = torch.where(kept[:, None, :, None], codes[src], codes[dst])
        if scales is not None:
            scales[dst] = torch.where(kept[:, None, None, :], scales[src], scales[dst])
    return {"table": s["table_out"], "copies": copies, **_held(c)}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        plain = {"rotate": _plain_rotate, "store": _plain_store, "extend": _plain_extend, "collect": _plain_collect,
                 "select": _plain_select, "reorder": _plain_reorder}
        return plain[op](s)
    fp4 = s["fp4"]
    if op == "rotate":
        q, k = fp4.qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], s["q_weight"], s["k_weight"],
                                eps=s["eps"], interleaved=case["interleaved"], dtype=s["q"].dtype)
        return {"q": q, "k": k}
    if op == "store":
        q = fp4.qk_norm_rope_append(s["handle"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freqs"],
                                    s["q_weight"], s["k_weight"], eps=s["eps"], interleaved=case["interleaved"])
        return {"q": q, **_held(s["cache"])}
    if op == "extend":
        plan = fp4.kv_pages_extend(s["pool"], s["table"], s["seq_lens"], s["new_lens"], s["tokens"], in_place=False)
        return {"slots": plan.slots, "positions": plan.positions, "cu_q": plan.cu_q, "cu_k": plan.cu_k,
                "seq_lens": plan.seq_lens, "table": s["table"], "state": plan.state}
    if op == "collect":
        fp4.kv_pages_collect(s["pool"], s["table"], s["seq_lens"])
        return {"free": s["free"], "count": s["state"][:1]}
    if op == "select":
        scores, parents, tokens = fp4.beam_select(s["logits"], s["scores"], k=case["k"], done=s["done"], end_token=END)
        return {"scores": scores, "parents": parents, "tokens": tokens}
    copies = fp4.kv_pages_reorder(s["table"], s["seq_lens"], s["parents"], case["page"], out=s["table_out"])
    fp4.kv_cache_copy(s["handle"], copies)
    return {"table": s["table_out"], "copies": copies, **_held(s["cache"])}


# ------------------------------------------------- the definition in 64 bits --

def _exact_rows(s, x):
    """Rows normed and rotated, float64, by complex numbers."""
    case, y = s["case"], s[x].double()
    if s["eps"] is not None:
        y = s[x + "_weight"].double() * y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + s["eps"])
    rot = case["rot"]
    if rot == 0:
        return y
    turn = torch.polar(torch.ones_like(s["freqs"]).expand(case["tokens"], -1), s["positions"].double()[:, None] * s["freqs"])
    head = y[..., :rot]
    pairs = head.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * turn[:, None])
    z = z if case["interleaved"] else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), y[..., rot:]], -1)


def _exact_reorder(s):
    """What the pages stand for after a reordering, group by group."""
    case, table = s["case"], s["table"].tolist()
    n = case["prompt"] + case["made"]
    at, off = n // case["page"], n % case["page"]
    got = {x: y.double() for x, y in _held(s["cache"]).items()}
    for b, parents in enumerate(s["parents"].tolist() if off else []):
        rows = table[b * case["beams"]:(b + 1) * case["beams"]]
        spare = [r for i, r in enumerate(rows) if i not in parents]
        further = [p for j, p in enumerate(parents) if p in parents[:j]]
        for p, heir in zip(further, spare):
            src, dst = rows[p][at], heir[at]
            for x, y in got.items():
                if x.endswith("scales"):
                    y[dst, ..., :off] = y[src, ..., :off]
                else:
                    y[dst, :, :off] = y[src, :, :off]
    return got


def exact(case, seed):
    op = case["op"]
    if op in ("extend", "collect"):
        return None  # whole numbers only
    s = prepare(case, seed)
    if op == "reorder":
        return {"table": None, "copies": None, **_exact_reorder(s)}
    if op == "rotate":
        return {"q": _exact_rows(s, "q"), "k": _exact_rows(s, "k")}
    if op == "store":
        got = {"q": _exact_rows(s, "q")}
        held, page = _held(s["cache"]), case["page"]
        kept = s["slots"] >= 0
        at, off = s["slots"][kept] // page, s["slots"][kept] % page
        for x, rows in (("k", _exact_rows(s, "k")), ("v", s["v"].double())):
            rows = rows[kept]
            got[x] = held[x].double()
            if case["fmt"] == "bf16":
                got[x][at, :, off] = rows
                continue
            b = rows.unflatten(-1, (-1, 32))
            top = torch.floor(torch.log2(b.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -119))) - 8
            got[x][at, :, off] = (b * torch.exp2(-top)).clamp(-448.0, 448.0).flatten(-2)  # before E4M3's rounding
            got[x + "_scales"] = held[x + "_scales"].double()
            got[x + "_scales"][at, :, :, off] = torch.exp2(top).squeeze(-1)
        return got
    z = s["logits"].double().view(case["batch"], case["beams"], -1)
    top = z.amax(-1, keepdim=True)
    total = z - top - torch.log(torch.exp(z - top).sum(-1, keepdim=True)) + s["scores"].double()[..., None]
    if s["done"] is not None:
        total[s["done"]] = -math.inf
        total[..., END] = torch.where(s["done"], s["scores"].double(), total[..., END])
    return {"scores": torch.topk(total.flatten(1), case["k"], dim=-1).values, "parents": None, "tokens": None}
