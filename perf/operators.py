"""Attention over a block-scaled key-value cache: what is measured.

Three operators of a serving step, each in a plain form (elementary torch operations in
32 bits) and as the library's own calls:

* ``store`` / ``restore``: new keys and values are quantized into a paged cache as they are
  written; ``restore`` then reads a whole context back as bf16, as the attention of a
  prompt's next chunk needs it.
* ``decode``: one new token of every sequence attends to its keys and values in the cache.
* ``prompt``: causal attention of whole prompts, packed one behind the other.

Cache layout (both forms): keys and values each as codes [pages, heads, page, row bytes]
(bf16: [pages, heads, page, head_dim]) and scale bytes [pages, heads, head_dim / block, page].
A slot is page * page_size + offset; a sequence's pages stand in its row of the block table,
unused entries of which are -1.
"""
import random

import torch

own = False

# block length along head_dim and bits a value, scales included
BLOCK = {"bf16": 0, "mxfp8": 32, "nvfp4": 16, "mxfp4": 32}
BITS = {"bf16": 16.0, "mxfp8": 8.25, "nvfp4": 4.5, "mxfp4": 4.25}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one chat user on an otherwise idle card: latency of one decode step of one layer
        {"name": "decode_one_bf16", "op": "decode", "fmt": "bf16", "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "batch": 1, "shortest": 517, "longest": 517, "window": 0, "lens": 0},
        # a small batch of short chats, some of its places empty (length 0), narrow heads, one key head each
        {"name": "decode_short_mxfp8", "op": "decode", "fmt": "mxfp8", "heads": 12, "kv_heads": 12, "dim": 64,
         "page": 16, "batch": 24, "shortest": 0, "longest": 300, "window": 0, "lens": 1},
        # a full serving batch of ragged lengths; heads of a 5120-wide layer
        {"name": "decode_batch_nvfp4", "op": "decode", "fmt": "nvfp4", "heads": 40, "kv_heads": 8, "dim": 128,
         "page": 64, "batch": 64, "shortest": 200, "longest": 16384, "window": 0, "lens": 2},
        # a few users with whole books in the context: one long axis, few rows
        {"name": "decode_long_mxfp4", "op": "decode", "fmt": "mxfp4", "heads": 32, "kv_heads": 4, "dim": 128,
         "page": 64, "batch": 3, "shortest": 90001, "longest": 131072, "window": 0, "lens": 3},
        # a layer that looks back only so far, wide heads, wide batch
        {"name": "decode_window_mxfp8", "op": "decode", "fmt": "mxfp8", "heads": 16, "kv_heads": 2, "dim": 256,
         "page": 32, "batch": 129, "shortest": 100, "longest": 8000, "window": 1024, "lens": 4},
        # a handful of one-line prompts that arrive together
        {"name": "prompt_lines", "op": "prompt", "heads": 8, "kv_heads": 2, "dim": 64, "batch": 5,
         "shortest": 1, "longest": 130, "context": 0, "window": 0, "lens": 5},
        # the prompts of several users in one packed batch
        {"name": "prompt_packed", "op": "prompt", "heads": 32, "kv_heads": 8, "dim": 128, "batch": 7,
         "shortest": 60, "longest": 1900, "context": 0, "window": 0, "lens": 6},
        # one long document; heads of a 5120-wide layer
        {"name": "prompt_document", "op": "prompt", "heads": 40, "kv_heads": 8, "dim": 128, "batch": 1,
         "shortest": 8192, "longest": 8192, "context": 0, "window": 0, "lens": 7},
        # the next chunk of a long prompt against what is in the cache already, in a windowed layer, wide heads
        {"name": "prompt_chunk_window", "op": "prompt", "heads": 16, "kv_heads": 4, "dim": 256, "batch": 2,
         "shortest": 777, "longest": 2048, "context": 5001, "window": 4096, "lens": 8},
        # one decode step's keys and values of a batch go into the cache
        {"name": "store_step_mxfp8", "op": "store", "fmt": "mxfp8", "kv_heads": 8, "dim": 128, "page": 64,
         "batch": 64, "shortest": 1, "longest": 1, "context": 700, "lens": 9},
        # a small chunk goes in, and its context comes back for the chunk's attention
        {"name": "restore_chunk_mxfp4", "op": "restore", "fmt": "mxfp4", "kv_heads": 2, "dim": 64, "page": 16,
         "batch": 3, "shortest": 33, "longest": 257, "context": 129, "lens": 10},
        # long prompts' chunks go in, their whole contexts come back
        {"name": "restore_prompt_nvfp4", "op": "restore", "fmt": "nvfp4", "kv_heads": 8, "dim": 128, "page": 64,
         "batch": 4, "shortest": 1500, "longest": 4096, "context": 12001, "lens": 11},
    ]


def _log(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prompt", "prompt", "store", "restore"])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 5, 8, 12])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while kv * group > 48:
        group = max(1, group // 2)
    case = {"op": op, "dim": dim, "kv_heads": kv, "lens": rng.randrange(1, 1 << 30)}
    if op != "prompt":
        case["fmt"] = rng.choice(["bf16", "mxfp8", "nvfp4", "mxfp4"])
        case["page"] = rng.choice([16, 32, 64, 128])
    if op == "store":
        case["fmt"] = rng.choice(["bf16", "mxfp8"])
    if op == "decode":
        case["heads"] = kv * group
        case["batch"] = _log(rng, 1, 192)
        # a padded batch holds no more than the largest listed one
        token = 2 * kv * dim * BITS[case["fmt"]] / 8
        case["longest"] = _log(rng, 1, min(131072, int(280e6 / token / case["batch"])))
        case["shortest"] = rng.choice([0, 1, case["longest"], _log(rng, 1, case["longest"])])
        case["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    elif op == "prompt":
        case["heads"] = kv * group
        case["batch"] = _log(rng, 1, 16)
        # all queries against all keys: no more than the largest listed case
        most = min(8192, int((37 * 8192 ** 2 * 128 / max(128, dim) / case["heads"]) ** 0.5))
        case["longest"] = _log(rng, 1, max(1, most // case["batch"]))
        case["shortest"] = rng.choice([1, case["longest"], _log(rng, 1, case["longest"])])
        case["context"] = rng.choice([0, 0, _log(rng, 1, 8192)])
        keys = case["batch"] * (case["longest"] + case["context"])
        while case["context"] and (case["batch"] * case["longest"] * keys > most ** 2 or keys > 16384):
            case["context"] //= 2
            keys = case["batch"] * (case["longest"] + case["context"])
        case["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    else:
        case["batch"] = _log(rng, 1, 128)
        most = int(300e6 / (8 * kv * dim) / case["batch"])
        case["longest"] = _log(rng, 1, min(8192, most // 2))
        case["shortest"] = rng.choice([1, case["longest"], _log(rng, 1, case["longest"])])
        case["context"] = rng.choice([0, _log(rng, 1, min(8192, most // 2))])
    return case


def _lengths(case):
    """The sequences' lengths: `longest` once, the others between the two, over the logarithm."""
    rng = random.Random(case["lens"])
    low, high = case["shortest"], case["longest"]
    lens = [high] + [max(low, _log(rng, max(low, 1), max(high, 1)) if rng.random() > 0.05 else low)
                     for _ in range(case["batch"] - 1)]
    rng.shuffle(lens)
    return lens


def _attended(case, lens):
    """Pairs of a query and a key it sees, over all sequences."""
    win, pairs = case["window"], 0
    for n in lens:
        if case["op"] == "decode":
            pairs += min(n, win) if win else n
        else:
            c = case["context"]  # query i sees i + c + 1 keys, or the window's last ones
            full = n if not win else max(0, min(n, win - c))
            pairs += full * c + full * (full + 1) // 2 + (n - full) * win
    return pairs


def work(case):
    lens, kv, dim = _lengths(case), case["kv_heads"], case["dim"]
    if case["op"] == "decode":
        keys = _attended(case, lens)
        rows = case["batch"] * case["heads"] * dim
        return {"bytes": 2 * keys * kv * dim * BITS[case["fmt"]] / 8 + 4 * rows,
                "flops": 4.0 * keys * case["heads"] * dim}
    if case["op"] == "prompt":
        q, k = sum(lens), sum(lens) + case["batch"] * case["context"]
        if case["window"]:
            k = sum(min(n + case["context"], n + case["window"] - 1) for n in lens)
        return {"bytes": 2.0 * dim * (2 * q * case["heads"] + 2 * k * kv) + 4.0 * q * case["heads"],
                "flops": 4.0 * _attended(case, lens) * case["heads"] * dim}
    new = 2 * sum(lens) * kv * dim
    n = {"bytes": new * (2 + BITS[case["fmt"]] / 8), "flops": 4.0 * new}
    if case["op"] == "restore":
        whole = new + 2 * case["batch"] * case["context"] * kv * dim
        # what was just written is read once more, with the context before it
        n = {"bytes": n["bytes"] + whole * (2 + BITS[case["fmt"]] / 8), "flops": n["flops"] + 2.0 * whole}
    return n


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _keys(g, shape):
    """Keys as a projection leaves them: normal, a few channels of every head much larger."""
    x = torch.randn(shape, device="cuda", generator=g)
    gain = torch.ones(shape[-2:], device="cuda")
    gain[torch.rand(shape[-2:], device="cuda", generator=g) < 0.03] = 6.0
    return (x * gain).to(torch.bfloat16)


def _cache(case, g, pages):
    """A cache with arbitrary contents: codes of all values, scales of the sizes that a
    quantizer gives for values around 1."""
    fmt, kv, page, dim = case["fmt"], case["kv_heads"], case["page"], case["dim"]
    c = {"fmt": fmt}
    for s in "kv":
        if fmt == "bf16":
            c[s + "_codes"] = torch.randn(pages, kv, page, dim, device="cuda", generator=g).to(torch.bfloat16)
            c[s + "_scales"] = c[s + "_tscale"] = None
            continue
        row = dim if fmt == "mxfp8" else dim // 2
        codes = torch.randint(0, 256, (pages, kv, page, row), device="cuda", generator=g, dtype=torch.uint8)
        shape = (pages, kv, dim // BLOCK[fmt], page)
        if fmt == "mxfp8":  # E4M3 bytes 0x7F and 0xFF are not numbers: 0x7E and 0xFE in their place
            codes = torch.where((codes & 127) == 127, codes - 1, codes)
            scales = torch.randint(118, 121, shape, device="cuda", generator=g, dtype=torch.uint8)
        elif fmt == "mxfp4":
            scales = torch.randint(125, 128, shape, device="cuda", generator=g, dtype=torch.uint8)
        else:
            scales = torch.randint(0x30, 0x48, shape, device="cuda", generator=g, dtype=torch.uint8)
        c[s + "_codes"], c[s + "_scales"], c[s + "_tscale"] = codes, scales, None
        if fmt == "nvfp4":
            c[s + "_tscale"] = 0.2 + 0.3 * torch.rand(kv, device="cuda", generator=g)
    return c


def _tables(case, lens, seed):
    """A block table over pages in random order, and the number of pages."""
    page = case["page"]
    need = [(n + page - 1) // page for n in lens]
    width, pages = max(1, max(need)), sum(need) + 3
    rows = torch.arange(width).unsqueeze(0).expand(len(lens), width)
    used = rows < torch.tensor(need).unsqueeze(1)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    table[used] = order[:sum(need)].to(torch.int32)
    return table, pages


def _offsets(lens):
    return torch.tensor([0] + lens).cumsum(0)


def prepare(case, seed):
    g, lens, dim = _gen(seed), _lengths(case), case["dim"]
    s = {"case": case, "lens": lens}
    if case["op"] == "decode":
        table, pages = _tables(case, lens, seed)
        s["cache"] = _cache(case, g, pages)
        s["q"] = (2.0 * torch.randn(case["batch"], case["heads"], dim, device="cuda", generator=g)).to(torch.bfloat16)
        s["table"] = table.cuda()
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    elif case["op"] == "prompt":
        q_offs, k_offs = _offsets(lens), _offsets([n + case["context"] for n in lens])
        tokens, keys = int(q_offs[-1]), int(k_offs[-1])
        s["q"] = _keys(g, (tokens, case["heads"], dim))
        s["k"] = _keys(g, (keys, case["kv_heads"], dim))
        s["v"] = torch.randn(keys, case["kv_heads"], dim, device="cuda", generator=g).to(torch.bfloat16)
        s["cu_q"], s["cu_k"] = q_offs.to(torch.int32).cuda(), k_offs.to(torch.int32).cuda()
        s["keys"] = keys
        s["lse"] = torch.empty(tokens, case["heads"], dtype=torch.float32, device="cuda")
    else:
        whole = [n + case["context"] for n in lens]
        table, pages = _tables(case, whole, seed)
        s["cache"] = _cache(case, g, pages)
        tokens, page = sum(lens), case["page"]
        # keys and values are columns of one projection's rows
        kv = _keys(g, (tokens, 2 * case["kv_heads"], dim))
        s["k"], s["v"] = kv[:, :case["kv_heads"]], kv[:, case["kv_heads"]:]
        seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
        at = torch.arange(tokens) - _offsets(lens)[seq] + case["context"]
        s["slots"] = (table[seq, at // page].long() * page + at % page).cuda()
        s["table"], s["cu"] = table.cuda(), _offsets(whole).to(torch.int32).cuda()
        s["tokens"] = sum(whole)
    if own:
        import block_scaled_fp4_04_amd as fp4

        s["fp4"] = fp4
        if "cache" in s:  # the handle that a program keeps
            s["handle"] = fp4.KVCache(**s["cache"])
    return s


# ------------------------------------------------------------- plain form --

def _e2m1(codes):
    """Packed bytes [..., n] -> the values [..., 2n] of their E2M1 codes, low nibble first."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    return grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]


def _values(c, s, codes, scales):
    """Codes [..., heads, page, row] and scale bytes [..., heads, blocks, page] -> fp32 [..., heads, page, dim]."""
    if c["fmt"] == "bf16":
        return codes.float()
    if c["fmt"] == "nvfp4":
        x, f = _e2m1(codes), scales.view(torch.float8_e4m3fn).float()
        f = f * c[s + "_tscale"][:, None, None]
    else:
        x = codes.view(torch.float8_e4m3fn).float() if c["fmt"] == "mxfp8" else _e2m1(codes)
        f = torch.exp2(scales.float() - 127.0)
    return x * f.transpose(-1, -2).repeat_interleave(BLOCK[c["fmt"]], -1)


def _gathered(c, s, table):
    """The padded contexts of a block table: fp32 [batch, heads, keys, dim]."""
    at = table.clamp(min=0).long()
    x = _values(c, s, c[s + "_codes"][at], None if c[s + "_scales"] is None else c[s + "_scales"][at])
    return x.transpose(1, 2).flatten(2, 3)


def _softmax(scores, seen, v):
    """Softmax of scores [..., queries, keys] where `seen`, times v; rows that see nothing give 0."""
    scores = scores.masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return out, (top + total.log()).squeeze(-1)


def _plain_decode(s):
    case, q = s["case"], s["q"].float()
    k, v = _gathered(s["cache"], "k", s["table"]), _gathered(s["cache"], "v", s["table"])
    batch, kv, keys, dim = k.shape
    scores = torch.matmul(q.view(batch, kv, -1, dim), k.transpose(-1, -2).contiguous()) * dim ** -0.5
    at, n = torch.arange(keys, device="cuda"), s["seq_lens"][:, None]
    seen = at < n
    if case["window"]:
        seen = seen & (at >= n - case["window"])
    out, _ = _softmax(scores, seen[:, None, None, :], torch.where(seen[:, None, :, None], v, 0.0))
    return out.reshape(q.shape).to(torch.bfloat16)


def _plain_prompt(s):
    case, q, k, v = s["case"], s["q"].float(), s["k"].float(), s["v"].float()
    tokens, heads, dim = q.shape
    keys, kv = k.shape[:2]
    qt = q.view(tokens, kv, heads // kv, dim).permute(1, 2, 0, 3).reshape(kv, -1, dim)
    scores = torch.matmul(qt, k.permute(1, 2, 0).contiguous()).mul_(dim ** -0.5).view(kv, heads // kv, tokens, keys)
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    iq, ik = torch.arange(tokens, device="cuda"), torch.arange(keys, device="cuda")
    bq, bk = torch.searchsorted(cu_q, iq, right=True) - 1, torch.searchsorted(cu_k, ik, right=True) - 1
    # positions within the sequence; the last query stands at the last key
    pq = iq - cu_q[bq + 1] + (cu_k[bq + 1] - cu_k[bq])
    pk = ik - cu_k[bk]
    seen = (bq[:, None] == bk) & (pk <= pq[:, None])
    if case["window"]:
        seen = seen & (pk > pq[:, None] - case["window"])
    out, lse = _softmax(scores, seen, v.transpose(0, 1).contiguous().unsqueeze(1))
    out = out.permute(2, 0, 1, 3).reshape(tokens, heads, dim).to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(2, 0, 1).reshape(tokens, heads).contiguous()}


def _quantized(c, s, x):
    """x fp32 [tokens, heads, dim] -> its codes [tokens, heads, row] and scale bytes [tokens, heads, blocks]."""
    b = x.unflatten(-1, (-1, BLOCK[c["fmt"]]))
    amax = b.abs().amax(-1, keepdim=True)
    if c["fmt"] == "nvfp4":
        t = c[s + "_tscale"][:, None, None]
        scale = (amax / (6.0 * t)).clamp(max=448.0).to(torch.float8_e4m3fn)
        step = scale.float() * t
        y = torch.where(step > 0, b / torch.where(step > 0, step, torch.ones_like(step)), b * 0.0)
        scale = scale.view(torch.uint8)
    else:  # the power of two that takes the block's largest value to the top binade of its type
        e = torch.frexp(amax).exponent - 1 - (8 if c["fmt"] == "mxfp8" else 2)
        e = torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))
        y = torch.ldexp(b, -e)
        scale = (e + 127).to(torch.uint8)
    if c["fmt"] == "mxfp8":
        codes = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    else:  # to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; of two as near, the one with the even code
        a = y.abs()
        m = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
        n = (m + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
        codes = n[..., 0::2] | (n[..., 1::2] << 4)
    return codes, scale.squeeze(-1)


def _plain_append(c, x, s, slots):
    page = c[s + "_codes"].shape[2]
    at, off = slots // page, slots % page
    if c["fmt"] == "bf16":
        c[s + "_codes"][at, :, off] = x
        return
    codes, scales = _quantized(c, s, x.float())
    c[s + "_codes"][at, :, off] = codes
    c[s + "_scales"].transpose(2, 3)[at, :, off] = scales


def _plain_read(c, s, table, cu, tokens):
    page = c[s + "_codes"].shape[2]
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cu.long(), t, right=True) - 1
    pos = t - cu[b]
    at, off = table[b, pos // page].long(), pos % page
    codes = c[s + "_codes"][at, :, off].unsqueeze(2)
    scales = None if c[s + "_scales"] is None else c[s + "_scales"].transpose(2, 3)[at, :, off].unsqueeze(3)
    return _values(c, s, codes, scales).squeeze(2).to(torch.bfloat16)


def _held(c):
    """What the cache holds: its values' and scales' types say what they stand for."""
    if c["fmt"] == "bf16":
        return {"k": c["k_codes"], "v": c["v_codes"]}
    return {"k": c["k_codes"].view(torch.float8_e4m3fn), "v": c["v_codes"].view(torch.float8_e4m3fn),
            "k_scales": c["k_scales"].view(torch.float8_e8m0fnu), "v_scales": c["v_scales"].view(torch.float8_e8m0fnu)}


def _plain(s):
    op, c = s["case"]["op"], s.get("cache")
    if op == "decode":
        return _plain_decode(s)
    if op == "prompt":
        return _plain_prompt(s)
    _plain_append(c, s["k"], "k", s["slots"])
    _plain_append(c, s["v"], "v", s["slots"])
    if op == "store":
        return _held(c)
    return {"k": _plain_read(c, "k", s["table"], s["cu"], s["tokens"]),
            "v": _plain_read(c, "v", s["table"], s["cu"], s["tokens"])}


def run(state):
    if not own:
        return _plain(state)
    s, fp4, case = state, state["fp4"], state["case"]
    if case["op"] == "decode":
        return fp4.attn_decode_paged(s["q"], s["handle"], s["table"], s["seq_lens"], window=case["window"])
    if case["op"] == "prompt":
        out = fp4.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=True, window=case["window"],
                               lse=s["lse"])
        return {"out": out, "lse": s["lse"]}
    fp4.kv_cache_append(s["handle"], s["k"], s["v"], s["slots"])
    if case["op"] == "store":
        return _held(s["cache"])
    k, v = fp4.kv_cache_read(s["handle"], s["table"], s["cu"], s["tokens"])
    return {"k": k, "v": v}


# ------------------------------------------------- the definition in 64 bits --

def _exact_rows(c, s, ids, heads, dim):
    """The cached rows of one sequence, float64 [heads, len(ids), dim], ids = (page, offset) of each."""
    at, off = ids
    codes = c[s + "_codes"][at, :, off].transpose(0, 1)
    if c["fmt"] == "bf16":
        return codes.double()
    scales = c[s + "_scales"][at, :, :, off].transpose(0, 1).long()
    if c["fmt"] == "mxfp8":
        n = codes.long()
        e, m = (n >> 3) & 15, (n & 7).double()
        x = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m * 2.0 ** -9)
        x = torch.where(n >= 128, -x, x)
    else:
        n = torch.empty(*codes.shape[:2], dim, dtype=torch.long, device=codes.device)
        n[..., 0::2], n[..., 1::2] = (codes & 15).long(), (codes >> 4).long()
        e, m = (n >> 1) & 3, (n & 1).double()
        x = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).double()), m / 2)
        x = torch.where(n >= 8, -x, x)
    if c["fmt"] == "nvfp4":
        e, m = (scales >> 3) & 15, (scales & 7).double()
        f = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m * 2.0 ** -9)
        f = f * c[s + "_tscale"].double()[:, None, None]
    else:
        f = torch.exp2((scales - 127).double())
    return (x.unflatten(-1, (f.shape[-1], -1)) * f.unsqueeze(-1)).flatten(-2)


def _exact_attention(q, k, v, first, last, dim):
    """One sequence: q [heads, queries, dim], k and v [kv heads, keys, dim], query i sees the keys
    first[i] .. last[i] - 1.  (out, lse), a head at a time."""
    group, outs, lses = q.shape[0] // k.shape[0], [], []
    at = torch.arange(k.shape[1], device=q.device)
    hidden = (at < first[:, None]) | (at >= last[:, None])
    for h in range(q.shape[0]):
        z = torch.matmul(q[h], k[h // group].t().contiguous()) / dim ** 0.5
        z[hidden] = float("-inf")
        lse = torch.logsumexp(z, -1)
        w = torch.exp(z - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[:, None])
        outs.append(torch.matmul(w, v[h // group]))
        lses.append(lse)
    return torch.stack(outs), torch.stack(lses)


def _exact_nearest(y, top):
    """y (float64, not above `top`) rounded to the grid of E4M3 (top 448) or E2M1 (top 6), ties to even."""
    low, bits = (-6, 3) if top == 448.0 else (0, 1)
    a = y.abs().clamp(max=top)
    e = torch.frexp(a).exponent - 1
    ulp = torch.exp2((e.clamp(min=low) - bits).double())
    return torch.sign(y) * (torch.round(a / ulp) * ulp).clamp(max=top)


def _exact_stored(c, s, x):
    """What x [tokens, heads, dim] stands for once it is stored: (elements, scales, values)."""
    if c["fmt"] == "bf16":
        return x.double(), None, x.double()
    b = x.double().unflatten(-1, (-1, BLOCK[c["fmt"]]))
    amax = b.abs().amax(-1, keepdim=True)
    if c["fmt"] == "nvfp4":
        t = c[s + "_tscale"].double()[:, None, None]
        f = _exact_nearest(amax / (6 * t), 448.0) * t
    else:
        e = torch.frexp(amax).exponent - 1 - (8 if c["fmt"] == "mxfp8" else 2)
        f = torch.exp2(torch.where(amax > 0, e.clamp(-127, 127), -127).double())
    n = torch.where(f > 0, b / torch.where(f > 0, f, 1.0), 0.0)
    n = _exact_nearest(n, 448.0 if c["fmt"] == "mxfp8" else 6.0)
    return n.flatten(-2), f.squeeze(-1), (n * f).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    lens, dim, c = s["lens"], case["dim"], s.get("cache")
    if case["op"] == "decode":
        page, out = case["page"], torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            first = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            pos = torch.arange(first, n, device="cuda")
            ids = s["table"][b].long()[pos // page], pos % page
            k = _exact_rows(c, "k", ids, case["kv_heads"], dim)
            v = _exact_rows(c, "v", ids, case["kv_heads"], dim)
            whole = torch.tensor([0], device="cuda"), torch.tensor([n - first], device="cuda")
            out[b] = _exact_attention(s["q"][b].double()[:, None], k, v, *whole, dim)[0][:, 0]
        return out
    if case["op"] == "prompt":
        outs, lses, q0, k0 = [], [], 0, 0
        for n in lens:
            keys = n + case["context"]
            last = torch.arange(n, device="cuda") + case["context"] + 1
            first = (last - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(last)
            o, l = _exact_attention(s["q"][q0:q0 + n].double().transpose(0, 1).contiguous(),
                                    s["k"][k0:k0 + keys].double().transpose(0, 1).contiguous(),
                                    s["v"][k0:k0 + keys].double().transpose(0, 1).contiguous(), first, last, dim)
            outs.append(o.transpose(0, 1))
            lses.append(l.t())
            q0, k0 = q0 + n, k0 + keys
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    page, got = case["page"], {}
    at, off = s["slots"] // page, s["slots"] % page
    for x in "kv":
        elements, scales, values = _exact_stored(c, x, s[x])
        if case["op"] == "store":
            held = _held(c)
            got[x] = held[x].double()
            got[x][at, :, off] = elements
            if scales is not None:
                got[x + "_scales"] = held[x + "_scales"].double()
                got[x + "_scales"][at, :, :, off] = scales
            continue
        rows, new = [], 0
        for b, n in enumerate(lens):
            pos = torch.arange(case["context"], device="cuda")
            ids = s["table"][b].long()[pos // page], pos % page
            rows.append(_exact_rows(c, x, ids, case["kv_heads"], dim).transpose(0, 1))
            rows.append(values[new:new + n])
            new += n
        got[x] = torch.cat(rows)
    return got
