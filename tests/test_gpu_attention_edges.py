"""Attention at the edges: sequences that end inside a tile before rows that are not numbers, values
that are not numbers in masked places, scores of any size, weights far below the largest one,
single-token buffers of any stride, and every part of the launch rules."""
import numpy as np
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu


def _fp4():
    import block_scaled_fp4_04_amd as fp4

    return fp4


def _cu(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_ends_before_nan(dim, causal):
    """Every second sequence's keys and values are NaN, and so is the memory behind the last one: rows of a
    tile past a sequence's end count as zeros wherever the end falls within the tile."""
    fp4 = _fp4()
    g = torch.Generator().manual_seed(dim)
    ends = [1, 5, 7, 8, 9, 15, 16, 17, 20, 24, 31, 32, 33, 40, 48, 63, 65, 1]
    lens = [n for e in ends for n in (e, 3)][:-1]
    n, heads, kv = sum(lens), 2, 1
    q, k, v = _randn(g, n, heads, dim), _randn(g, n + 70, kv, dim), _randn(g, n + 70, kv, dim)
    offs = np.cumsum([0] + lens)
    for b in range(1, len(lens), 2):
        k[offs[b]:offs[b + 1]] = v[offs[b]:offs[b + 1]] = float("nan")
    k[n:] = v[n:] = float("nan")
    lse = torch.empty(n, heads, device="cuda")
    out = fp4.attn_prefill(q.cuda(), k.cuda()[:n], v.cuda()[:n], _cu(lens), _cu(lens), causal=causal, dtype=torch.float32, lse=lse)
    for b in range(0, len(lens), 2):
        at = slice(offs[b], offs[b + 1])
        m = lens[b]
        last = [i + 1 if causal else m for i in range(m)]
        want = ref.attention(q[at].double(), k[at].double(), v[at].double(), dim ** -0.5, [0] * m, last)
        ref.check(out[at], lse[at], want, dim, 2.0 ** -8, f"{m} keys before NaN, head_dim {dim}")


def test_one_token_of_head_major_buffers():
    """A single query and key as views of large head-major buffers (their token stride is never followed)."""
    fp4 = _fp4()
    heads, dim = 8, 128
    q, k, v = (torch.randn(heads, 32768, dim, device="cuda").to(torch.bfloat16)[:, 5:6].transpose(0, 1) for _ in range(3))
    hold = torch.zeros(heads, 32768, dim, device="cuda", dtype=torch.bfloat16)
    out = hold[:, 7:8].transpose(0, 1)
    fp4.attn_prefill(q, k, v, _cu([1]), _cu([1]), out=out)
    assert torch.equal(out, v) and int((hold != 0).any(-1).sum()) == heads
    c = fp4.KVCache.alloc("bf16", 2, heads, 16, dim)
    fp4.kv_cache_append(c, k, v, torch.tensor([19], dtype=torch.int64, device="cuda"))
    table, one = torch.tensor([[1]], dtype=torch.int32, device="cuda"), torch.tensor([4], dtype=torch.int32, device="cuda")
    c.k_codes[1, :, :3], c.v_codes[1, :, :3] = c.k_codes[1, :, 3:4], c.v_codes[1, :, 3:4]
    assert torch.equal(fp4.attn_decode_paged(q, c, table, one), v)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("n", [1000, 20000])
def test_decode_weights_far_below_the_largest(fmt, n):
    """Every eighth key takes nearly all of the weight and has zeros as its values; the others, about 2^-26 of
    it each, make the whole output.  f16 weights stand 2^7 above 1, so one below 2^-14 is off by at most 2^-25,
    which is 2^-32 of the largest weight; the sum of the weights is n / 8 largest ones.  bf16 ones keep their range."""
    fp4 = _fp4()
    g = torch.Generator().manual_seed(n)
    dim, page = 64, 64
    k, v = torch.zeros(n, 1, dim), torch.rand(n, 1, dim, generator=g) + 0.5
    k[:, 0, 0] = 1.2 + 0.6 * torch.rand(n, generator=g)
    k[::8, 0, 0], v[::8] = 6.0, 0.0
    ts = torch.tensor([1.0 / 64]) if fmt == "nvfp4" else None
    pages = (n + page - 1) // page
    c = fp4.KVCache.alloc(fmt, pages, 1, page, dim, "cuda", *([None] * 2 if ts is None else [ts.cuda()] * 2))
    fp4.kv_cache_append(c, k.cuda(), v.cuda(), torch.arange(n, device="cuda"))
    t = None if ts is None else ts.numpy()
    kk, vv = (torch.from_numpy(ref.decode_rows(fmt, *ref.encode_rows(fmt, x.numpy(), t), t)) for x in (k, v))
    q = torch.zeros(1, 2, dim)
    q[0, :, 0] = torch.tensor([4.0, 4.125])
    q = q.to(torch.bfloat16)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lse = torch.empty(1, 2, device="cuda")
    out = fp4.attn_decode_paged(q.cuda(), c, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0,
                                dtype=torch.float32, lse=lse)
    want = ref.attention(q.double(), kk, vv, 1.0, [0], [n])
    half = fmt == "nvfp4"
    small = 2.0 ** -8 * vv.abs().sum(0)[None] / (n / 8)  # (the check takes 2^-24 of it)
    ref.check(out, lse, want, dim, 2.0 ** -11 if half else 2.0 ** -8, f"{fmt} {n}", small if half else None)


FAR = [3e5, 2e6, 1e9, 1e15, 1e30]


def _far_data(n, seed):
    """Keys of small whole scores with q = 1 or -1, so that every score is exact and the largest ones share all the weight."""
    g = torch.Generator().manual_seed(seed)
    k, v = torch.zeros(n, 1, 64), torch.randn(n, 1, 64, generator=g)
    k[:, 0, 0] = torch.tensor([-3.0, -2.0, -1.0, 0.5, 1.0, 2.0, 3.0, 4.0])[torch.randint(0, 8, (n,), generator=g)]
    k[torch.randperm(n, generator=g)[:3], 0, 0] = 6.0
    return k, v


def _far_want(q, k, v, scale, last):
    """The mean of the values whose scores are the largest, and the logarithm.  (Scores are compared before they are
    scaled: at 1e15 even 64 bits would round the logarithm of a weight.)"""
    out, lse = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    for i in range(q.shape[0]):
        for h in range(q.shape[1]):
            z = k[:last[i], 0] @ q[i, h]
            top = z == z.max()
            out[i, h], lse[i, h] = v[:last[i], 0][top].mean(0), z.max() * scale + float(top.sum().double().log())
    return out, lse


def _check_far(out, lse, want, v, what):
    """The largest scores' weights are equal, so they round alike; the rest is fp32 sums of at most 2^13 terms."""
    d = (out.cpu().double() - want[0]).abs()
    assert float(d.max()) <= (2.0 ** -8 + 2.0 ** -11) * float(v.abs().max()), f"{what}: {float(d.max())}"
    assert bool(((lse.cpu().double() - want[1]).abs() <= 2.0 ** -20 * want[1].abs()).all()), what


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("n", [700, 5000])
def test_decode_scores_far_out(fmt, n):
    """Scores up to the documented scale of 1e30: the largest take all of the weight, however they are rounded."""
    fp4 = _fp4()
    k, v = _far_data(n, n)
    ts = torch.tensor([1.0 / 64]) if fmt == "nvfp4" else None
    pages = (n + 63) // 64
    c = fp4.KVCache.alloc(fmt, pages, 1, 64, 64, "cuda", *([None] * 2 if ts is None else [ts.cuda()] * 2))
    fp4.kv_cache_append(c, k.cuda(), v.cuda(), torch.arange(n, device="cuda"))
    if fmt == "bf16":
        kk, vv = (x.to(torch.bfloat16).double() for x in (k, v))
    else:
        t = None if ts is None else ts.numpy()
        kk, vv = (torch.from_numpy(ref.decode_rows(fmt, *ref.encode_rows(fmt, x.numpy(), t), t)) for x in (k, v))
    q = torch.zeros(1, 2, 64)
    q[0, :, 0] = torch.tensor([1.0, -1.0])
    q = q.to(torch.bfloat16)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    for scale in FAR:
        lse = torch.empty(1, 2, device="cuda")
        out = fp4.attn_decode_paged(q.cuda(), c, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale,
                                    dtype=torch.float32, lse=lse)
        _check_far(out, lse, _far_want(q.double(), kk, vv, float(np.float32(scale)), [n]), vv, f"{fmt} {n} {scale}")


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_scores_far_out(dim):
    """The same for prompts: one of a few rows (keys split among workgroups) and one of many."""
    fp4 = _fp4()
    for lq, n in ((3, 5000), (300, 300)):
        k, v = (torch.nn.functional.pad(x, (0, dim - 64)).to(torch.bfloat16) for x in _far_data(n, n + dim))
        q = torch.zeros(lq, 2, dim)
        q[:, :, 0] = torch.tensor([1.0, -1.0])
        q = q.to(torch.bfloat16)
        for scale in FAR:
            lse = torch.empty(lq, 2, device="cuda")
            out = fp4.attn_prefill(q.cuda(), k.cuda(), v.cuda(), _cu([lq]), _cu([n]), scale=scale, dtype=torch.float32, lse=lse)
            want = _far_want(q.double(), k.double(), v.double(), float(np.float32(scale)), [i + 1 + n - lq for i in range(lq)])
            _check_far(out, lse, want, v.double(), f"{dim} {lq} {n} {scale}")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lq,lk,window", [(130, 130, 0), (200, 200, 70), (5, 6000, 0), (3, 5000, 900), (600, 1000, 333), (20, 9, 0)])
def test_prompt_values_that_are_not_numbers_where_masked(dim, lq, lk, window):
    """Infinities and NaN in V reach exactly the rows and columns that see them: later tokens' and those behind the window
    leave a row's bits as they are."""
    fp4 = _fp4()
    g = torch.Generator().manual_seed(dim + lk)
    heads, kv = 4, 2
    q, k, v = _randn(g, lq, heads, dim), _randn(g, lk, kv, dim), _randn(g, lk, kv, dim)
    pos = torch.arange(lq) + lk - lq
    at = sorted({lk - 1, lk - 2, lk - lq // 2 - 1, max(0, lk - lq), max(0, lk - lq - window), lk // 2 if window else lk - 1, 0})
    bad = v.clone()
    for i, key in enumerate(at):
        bad[key, i % kv, 7 * i % dim] = (float("inf"), float("-inf"), float("nan"))[i % 3]
        bad[key, (i + 1) % kv, (7 * i + 1) % dim] = (float("nan"), float("inf"), float("-inf"))[i % 3]
    run = lambda v: fp4.attn_prefill(q.cuda(), k.cuda(), v.cuda(), _cu([lq]), _cu([lk]), window=window, dtype=torch.float32,  # noqa: E731
                                     lse=lse).cpu()
    lse = torch.empty(lq, heads, device="cuda")
    clean = run(v)
    lse_clean = lse.clone()
    got = run(bad)
    assert torch.equal(lse, lse_clean)
    # what a row sees of them, by column: sums of infinities and NaN alone
    keys = torch.arange(lk)
    seen = keys <= pos[:, None]
    if window:
        seen &= keys > pos[:, None] - window
    hit = torch.where(torch.isfinite(bad), 0.0, bad.float())
    want = torch.zeros(lq, kv, dim)
    for key in at:
        want[seen[:, key]] += hit[key]
    want = want.repeat_interleave(heads // kv, 1)
    fine = want == 0
    assert torch.equal(got[fine], clean[fine])
    assert torch.equal(torch.nan_to_num(got[~fine], nan=1.0, posinf=2.0, neginf=3.0), torch.nan_to_num(want[~fine], nan=1.0, posinf=2.0, neginf=3.0))


def _attention_on_gpu(q, k, v, scale, first, last):
    """attention_ref.attention for long sequences: the same terms, a head at a time in float64 on the device."""
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    at = torch.arange(k.shape[0], device="cuda")
    hidden = (at < first[:, None]) | (at >= last[:, None])
    out, lse, mass, size = [], [], [], []
    for h in range(heads):
        kk, vv = k[:, h // group].double().contiguous(), v[:, h // group].double().contiguous()
        qq = q[:, h].double().contiguous()
        z = (qq @ kk.t().contiguous() * scale).masked_fill_(hidden, -float("inf"))
        lse.append(torch.logsumexp(z, 1))
        p = torch.exp(z - torch.where(torch.isinf(lse[-1]), 0.0, lse[-1])[:, None])
        out.append(p @ vv)
        mass.append(p @ vv.abs())
        size.append((qq.abs() @ kk.abs().t().contiguous() * scale).masked_fill_(hidden, 0.0).amax(1))
    return [torch.stack(x, 1).cpu() for x in (out, lse, mass, size)]


def _check_prompt(lq, lk, heads, kv, dim, window=0, causal=True, seed=0):
    fp4 = _fp4()
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = (torch.randn(n, h, dim, device="cuda", generator=g).to(torch.bfloat16) for n, h in ((sum(lq), heads), (sum(lk), kv), (sum(lk), kv)))
    lse = torch.full((sum(lq), heads), 7.0, device="cuda")
    out = fp4.attn_prefill(q, k, v, _cu(lq), _cu(lk), causal=causal, window=window, dtype=torch.float32, lse=lse)
    a = b = 0
    for n, m in zip(lq, lk):
        if n:
            pos = torch.arange(n, device="cuda") + m - n
            last = (pos + 1 if causal else torch.full_like(pos, m)).clamp(min=0)
            first = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
            want = _attention_on_gpu(q[a:a + n], k[b:b + m], v[b:b + m], dim ** -0.5, first, last) if m else \
                [torch.zeros(n, heads, dim, dtype=torch.float64), torch.full((n, heads), -float("inf"), dtype=torch.float64),
                 torch.zeros(n, heads, dim, dtype=torch.float64), torch.zeros(n, heads, dtype=torch.float64)]
            ref.check(out[a:a + n], lse[a:a + n], want, dim, 2.0 ** -8, f"{n} of {m}, {heads}/{kv}x{dim} window {window} causal {causal}")
        a, b = a + n, b + m


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_parts_by_row_tile(dim):
    """Row tiles of one call with different numbers of parts: none, one, as many as the call has; lengths
    around a part; windows that leave one part of many keys."""
    need = _fp4().lib().attn_prefill_workspace
    for lq, lk, window, heads, kv in (([3, 40, 1, 7, 2], [3000, 40, 447, 448, 449], 0, 4, 2), ([5, 5], [9000, 895], 0, 8, 2),
                                      ([300, 5, 0, 1], [3000, 60, 0, 897], 0, 4, 1), ([64, 9], [5000, 4000], 600, 4, 2),
                                      ([64, 9], [5000, 4000], 2000, 4, 2), ([20, 1], [9, 4000], 0, 2, 1)):
        assert need(sum(lq), heads, sum(lk), kv, dim, len(lq)) > 0
        _check_prompt(lq, lk, heads, kv, dim, window, seed=dim + sum(lk))
    _check_prompt([3, 40, 2], [3000, 40, 449], 4, 2, dim, causal=False, seed=dim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,heads,kv", [([7001], 6, 2), ([2500, 1, 0, 2300, 33, 1900], 6, 2), ([3100, 2700], 8, 8), ([8400], 8, 8)])
def test_prompt_tile_order(dim, lens, heads, kv):
    """Row tiles that fill the chip once and part of a second time: the second half comes in reverse (every row is checked).
    [8400] has more than that, so they come in order."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = sum(-(-n * heads // kv // 128) for n in lens)
    assert -(-cus // kv) < tiles and (tiles * kv <= 2 * cus or lens == [8400])
    assert _fp4().lib().attn_prefill_workspace(sum(lens), heads, sum(lens), kv, dim, len(lens)) == 0
    _check_prompt(lens, lens, heads, kv, dim, seed=len(lens))


def test_decode_more_rows_than_a_launch_holds():
    """2^20 + 3 sequences of 8 heads: more workgroups of 512 threads than one launch may have."""
    fp4 = _fp4()
    n, heads, dim = (1 << 20) + 3, 8, 64
    g = torch.Generator().manual_seed(0)
    c = fp4.KVCache.alloc("bf16", 1, heads, 16, dim)
    k, v = (_randn(g, 16, heads, dim).cuda() for _ in range(2))
    fp4.kv_cache_append(c, k, v, torch.arange(16, device="cuda"))
    q = _randn(g, 1, heads, dim).cuda()
    some = torch.arange(17, dtype=torch.int32, device="cuda")
    small = fp4.attn_decode_paged(q.expand(17, -1, -1), c, torch.zeros(17, 1, dtype=torch.int32, device="cuda"), some)
    lens = torch.randint(0, 17, (n,), generator=g, dtype=torch.int32).cuda()
    out = fp4.attn_decode_paged(q.expand(n, -1, -1), c, torch.zeros(n, 1, dtype=torch.int32, device="cuda"), lens)
    assert torch.equal(out.view(n, -1), small.view(17, -1)[lens.long()])


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_decode_many_sequences_of_wide_tables(fmt):
    """A batch with more sequences than a quarter of its table's keys takes a workgroup a row, at any length."""
    from test_gpu_attention import _check_decode

    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 30, 530)] + [1300, 0, 2047]
    _check_decode(fmt, lens, 2, 1, 64, 16, seed=21)


@pytest.mark.parametrize("count", [256, 257, 4500])
def test_prompt_sequences_by_search(count):
    """Batches of many sequences find their row tiles by search: empty ones between, some of several tiles, at the end too."""
    rng = np.random.default_rng(count)
    lq = [int(x) for x in rng.integers(0, 4, count)]
    for i in (0, 7, count // 2, count - 1):
        lq[i] = 200 + i % 50
    lk = [n + int(x) if n else 0 for n, x in zip(lq, rng.integers(0, 3, count))]
    fp4 = _fp4()
    g = torch.Generator(device="cuda").manual_seed(count)
    heads, kv, dim = 6, 2, 64
    q, k, v = (torch.randn(n, h, dim, device="cuda", generator=g).to(torch.bfloat16) for n, h in ((sum(lq), heads), (sum(lk), kv), (sum(lk), kv)))
    lse = torch.empty(sum(lq), heads, device="cuda")
    out = fp4.attn_prefill(q, k, v, _cu(lq), _cu(lk), dtype=torch.float32, lse=lse)
    # the same sequences, 100 a call
    oq, ok = np.cumsum([0] + lq), np.cumsum([0] + lk)
    for b in range(0, count, 100):
        e = min(b + 100, count)
        some = torch.empty(int(oq[e] - oq[b]), heads, device="cuda")
        part = fp4.attn_prefill(q[oq[b]:oq[e]], k[ok[b]:ok[e]], v[ok[b]:ok[e]], _cu(lq[b:e]), _cu(lk[b:e]), dtype=torch.float32, lse=some)
        assert torch.equal(out[oq[b]:oq[e]], part) and torch.equal(lse[oq[b]:oq[e]], some), b
    b = count // 2
    _check_prompt(lq[b - 5:b + 5], lk[b - 5:b + 5], heads, kv, dim)


def test_prompt_more_rows_than_a_launch_holds():
    """2^20 + 5 sequences of 8 heads: more workgroups of 256 threads than one launch of this kernel takes."""
    fp4 = _fp4()
    n, heads, dim = (1 << 20) + 5, 8, 64
    g = torch.Generator().manual_seed(1)
    q, k, v = (_randn(g, 1, heads, dim).cuda().expand(n, -1, -1) for _ in range(3))
    out = torch.full((n, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    fp4.attn_prefill(q, k, v, cu, cu, out=out)
    assert torch.equal(out, v)


# ---- the split form of decode: rows shared by workgroups, and the launch that joins them

def _split(lens, heads, kv, page, dim, slack=1):
    """The workspace of a call as _check_decode makes it: rows are split only where it is not empty."""
    fp4 = _fp4()
    width = max(1, max((n + page - 1) // page for n in lens)) + slack
    sizes = fp4._KvCacheArg(0, 1, kv, page, dim)
    import ctypes

    assert 4 * len(lens) < width * page  # (more sequences take a workgroup a row)
    return fp4.lib().attn_decode_paged_workspace(len(lens), heads, ctypes.byref(sizes), width)


def _check_split(fmt, lens, heads, kv, dim, page, **kw):
    from test_gpu_attention import _check_decode

    assert _split(lens, heads, kv, page, dim) > 0
    return _check_decode(fmt, lens, heads, kv, dim, page, **kw)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_decode_split_head_dims(fmt, dim):
    _check_split(fmt, [1500, 0, 1, 2333], 4, 2, dim, 64, seed=dim)


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
@pytest.mark.parametrize("count,longest", [(65, 1100), (129, 1500), (200, 1300), (257, 2000)])
def test_decode_split_many_sequences(fmt, count, longest):
    """More sequences than lanes of a wave, ragged, empty ones among them, the longest first, last and in the middle."""
    rng = np.random.default_rng(count)
    lens = [int(x) for x in rng.integers(0, 90, count)]
    for i in (0, 63, 64, count // 2, count - 1):
        lens[i] = longest - i
    _check_split(fmt, lens, 2, 1, 64, 16, seed=count)


@pytest.mark.parametrize("count,heads,kv", [(3, 17, 1), (2, 40, 1), (66, 40, 2), (130, 16, 1), (70, 20, 4)])
def test_decode_split_head_tiles(count, heads, kv):
    """Several tiles of 16 heads on a key head; more than 1024 rows to join, and fewer."""
    rng = np.random.default_rng(heads)
    lens = [int(x) for x in rng.integers(0, 60, count)]
    lens[count // 2], lens[-1] = 1777, 1025
    _check_split("mxfp4", lens, heads, kv, 64, 32, seed=count)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("window", [1000, 1100, 2999, 3001])
def test_decode_split_window(fmt, window):
    """Windows that start inside a tile of a row that several workgroups share (and one just under the split form)."""
    _check_split(fmt, [5003, 1100, 0, 2, 3000], 2, 1, 64 if window < 2000 else 128, 64, window=window, seed=window)


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("dim,window", [(64, 1024), (256, 1001), (128, 2069)])
def test_decode_window_fills_the_chip(fmt, dim, window):
    """Enough windowed rows take one workgroup each, though the table is wide."""
    count = -(-torch.cuda.get_device_properties(0).multi_processor_count // 8)
    rng = np.random.default_rng(dim)
    lens = [int(x) for x in rng.integers(0, 200, count)]
    lens[1], lens[2], lens[-1] = 2600, window + 1, window
    _check_split(fmt, lens, 8, 8, dim, 64, window=window, seed=window)


def test_decode_split_repeats_streams_graph():
    """The split form gives the same bits on every call, on another stream, with a caller's workspace of any contents, and
    from a captured graph whose lengths and queries change between replays."""
    fp4 = _fp4()
    from test_gpu_attention import _filled

    lens = [2900, 5, 0, 1333]
    c, table, _, _ = _filled(fp4, "nvfp4", lens, 2, 128, 16, 13)
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):  # unused bytes: numbers
        t[t == 255] = 0x31
    q = torch.randn(4, 8, 128, device="cuda").to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = fp4.attn_decode_paged_workspace(c, 4, 8, table.shape[1])
    assert ws.numel() > 0
    first = fp4.attn_decode_paged(q, c, table, n)
    assert torch.equal(first, fp4.attn_decode_paged(q, c, table, n))
    for fill in (0, 255):
        ws.fill_(fill)
        assert torch.equal(first, fp4.attn_decode_paged(q, c, table, n, workspace=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fp4.attn_decode_paged(q, c, table, n)
    side.synchronize()
    assert torch.equal(first, other)
    out, lse = torch.empty_like(q), torch.empty(4, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4.attn_decode_paged(q, c, table, n, out=out, lse=lse, workspace=ws)
    for step in range(4):
        q.copy_(torch.randn(4, 8, 128, device="cuda").to(torch.bfloat16))
        n.copy_(torch.tensor([2900 - 650 * step, 5 + step, step, 1333], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        again = torch.empty_like(lse)
        assert torch.equal(out, fp4.attn_decode_paged(q, c, table, n, lse=again)), step
        assert torch.equal(lse, again), step


def test_decode_split_parts_join_by_lse():
    """Windowed and whole results of split rows agree through the logarithms of their sums."""
    fp4 = _fp4()
    from test_gpu_attention import _filled

    c, table, k, v = _filled(fp4, "bf16", [3500], 1, 64, 16, 14)
    assert fp4.attn_decode_paged_workspace(c, 1, 4, table.shape[1]).numel() > 0
    q = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    lse = [torch.empty(1, 4, device="cuda") for _ in range(3)]
    n = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    whole = fp4.attn_decode_paged(q, c, table, n(3500), lse=lse[0], dtype=torch.float32)
    head = fp4.attn_decode_paged(q, c, table, n(1377), lse=lse[1], dtype=torch.float32)
    tail = fp4.attn_decode_paged(q, c, table, n(3500), window=3500 - 1377, lse=lse[2], dtype=torch.float32)
    assert torch.allclose(torch.logaddexp(lse[1], lse[2]), lse[0], atol=2e-6)
    w = [torch.exp(x - lse[0])[..., None] for x in lse[1:]]
    assert float((w[0] * head + w[1] * tail - whole).abs().max()) < 3 * 2.0 ** -8 * float(v.abs().max())


def test_decode_split_bad_ids_and_lengths_stay_inside():
    """As the one-launch form: page ids outside the cache and lengths outside the table are clamped."""
    fp4 = _fp4()
    c = fp4.KVCache.alloc("bf16", 5, 1, 64, 64)
    for t in (c.k_codes, c.v_codes):
        t.fill_(1.0)
    table = torch.randint(-(2 ** 31), 2 ** 31 - 1, (2, 40), dtype=torch.int64, device="cuda").to(torch.int32)
    n = torch.tensor([10 ** 9, -3], dtype=torch.int32, device="cuda")
    q = torch.ones(2, 1, 64, device="cuda", dtype=torch.bfloat16)
    assert fp4.attn_decode_paged_workspace(c, 2, 1, 40).numel() > 0
    out = fp4.attn_decode_paged(q, c, table, n)
    assert bool((out[0] == 1).all()) and bool((out[1] == 0).all())


def test_decode_split_values_that_are_not_numbers_where_masked():
    """Keys and values behind the window and past the end may hold anything."""
    fp4 = _fp4()
    n, window, dim = 3001, 1203, 128
    g = torch.Generator().manual_seed(3)
    k, v = _randn(g, 3072, 1, dim), _randn(g, 3072, 1, dim)
    c = fp4.KVCache.alloc("bf16", 48, 1, 64, dim)
    table = torch.arange(48, dtype=torch.int32, device="cuda")[None]
    assert fp4.attn_decode_paged_workspace(c, 1, 3, 48).numel() > 0
    q = _randn(g, 1, 3, dim).cuda()
    outs = []
    for spoil in (False, True):
        if spoil:
            k[:n - window], v[:n - window] = float("nan"), float("inf")
            k[n:], v[n:] = float("inf"), float("nan")
        fp4.kv_cache_append(c, k.cuda(), v.cuda(), torch.arange(3072, device="cuda"))
        outs.append(fp4.attn_decode_paged(q, c, table, torch.tensor([n], dtype=torch.int32, device="cuda"), window=window))
    assert torch.equal(outs[0], outs[1]) and bool(outs[0].isfinite().all())


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_layer_with_long_context(fmt):
    """The example layer with contexts whose decode step is split and captured with its workspace."""
    import importlib.util
    import os

    import test_gpu_attention_layer as layer

    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(layer.ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    worst, _, y = m.run(fmt, prompts=(1300, 17), steps=4)
    assert y.shape == (2, 1024) and bool(y.isfinite().all())
    assert worst < layer.BOUND[fmt], (fmt, worst)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_decode_every_scale_byte(fmt):
    """One key a sequence and a query of zeros, so that its value is the output, bit for bit: every finite block scale, as
    the cache is read back (below 2^-126 the 16-bit operands of the products may lose bits)."""
    fp4 = _fp4()
    dim, page = 64, 16
    top = 0x7E if fmt == "nvfp4" else 254 if fmt == "mxfp4" else 245  # the largest with finite values
    pages = -(-(top + 1) // page)
    ts = [torch.tensor([0.75], device="cuda")] * 2 if fmt == "nvfp4" else [None] * 2
    c = fp4.KVCache.alloc(fmt, pages, 1, page, dim, "cuda", *ts)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, device="cuda", generator=g, dtype=torch.uint8))
        if fmt == "mxfp8":
            t[(t & 127) == 127] = 0x7E
    c.k_scales.fill_(0x38 if fmt == "nvfp4" else 120)
    c.v_scales.copy_(torch.arange(pages * page, device="cuda").clamp(max=top).view(pages, 1, 1, page).expand_as(c.v_scales).to(torch.uint8))
    n = top + 1
    # every key is the last of a sequence of its own, behind a window of one
    at = torch.arange(n, device="cuda")
    table = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = (at // page).int()
    q = torch.zeros(n, 1, dim, device="cuda", dtype=torch.bfloat16)
    out = fp4.attn_decode_paged(q, c, table, (at % page + 1).int(), window=1, dtype=torch.float32)
    _, v = fp4.kv_cache_read(c, torch.arange(pages, dtype=torch.int32, device="cuda")[None], _cu([n]), n, dtype=torch.float32)
    wrong = (out[:, 0].double() - v[:, 0].double()).abs() > 2.0 ** -126
    assert not bool(wrong.any()), (fmt, wrong.nonzero()[:4].tolist())


def test_prompt_strides_past_4_gib():
    """Keys and values whose rows lie 16 MiB apart: offsets within the buffer pass 2^32 bytes."""
    fp4 = _fp4()
    n, dim, step = 300, 64, 1 << 23
    hold = torch.zeros(n * step, dtype=torch.bfloat16, device="cuda")
    k = hold.as_strided((n, 2, dim), (step, dim, 1))
    v = hold.as_strided((n, 2, dim), (step, dim, 1), 4 * dim)
    q, a, b = (torch.randn(n, h, dim, device="cuda").to(torch.bfloat16) for h in (4, 2, 2))
    k.copy_(a)
    v.copy_(b)
    assert torch.equal(fp4.attn_prefill(q, k, v, _cu([n]), _cu([n])), fp4.attn_prefill(q, a, b, _cu([n]), _cu([n])))


@pytest.mark.parametrize("empty", [3, 8, 9, 70, 30000])
def test_read_between_empty_sequences(empty):
    """Runs of empty sequences between the tokens of one tile, before the first and after the last."""
    fp4 = _fp4()
    lens = [0] * empty + [5] + [0] * empty + [1, 2] + [0] * empty + [40] + [0] * empty
    used = [i for i, n in enumerate(lens) if n]
    c = fp4.KVCache.alloc("bf16", 6, 2, 16, 64)
    table = torch.full((len(lens), 3), -1, dtype=torch.int32)
    pages, slots = iter(range(6)), []
    for i in used:
        for j in range((lens[i] + 15) // 16):
            table[i, j] = next(pages)
        slots += [int(table[i, p // 16]) * 16 + p % 16 for p in range(lens[i])]
    n = sum(lens)
    k, v = (torch.randn(n, 2, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    fp4.kv_cache_append(c, k, v, torch.tensor(slots, dtype=torch.int64, device="cuda"))
    kr, vr = fp4.kv_cache_read(c, table.cuda(), _cu(lens), n + 3)
    assert torch.equal(kr[:n], k) and torch.equal(vr[:n], v)
    assert not bool(kr[n:].any()) and not bool(vr[n:].any())
