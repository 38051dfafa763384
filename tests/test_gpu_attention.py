"""Decode attention over the paged cache and attention of packed prompts against plain 64-bit
references: every format and head layout, lengths around tiles and pages, empty rows, windows,
strides, values that are not numbers where nothing may look, streams and graphs."""
import numpy as np
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

FMTS = ["bf16", "mxfp8", "nvfp4", "mxfp4"]
WEIGHT_ULP = {"bf16": 2.0 ** -8, "mxfp8": 2.0 ** -8, "mxfp4": 2.0 ** -8, "nvfp4": 2.0 ** -11}


def _fp4():
    import block_scaled_fp4_04_amd as fp4

    return fp4


def _filled(fp4, fmt, lens, kv_heads, dim, page, seed, spread=1.0):
    """A cache whose unused bytes read as NaN (or as garbage where the type has none), the block table
    with unusable entries past the pages in use, and the keys and values it holds (float64)."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    pages, width = sum(need) + 2, max(1, max(need)) + 1
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), width), 2 ** 30 + 1, dtype=torch.int32)
    table[::2] = -7
    slots = []
    for b, n in enumerate(lens):
        for i in range(need[b]):
            table[b, i] = order.pop()
        slots += [int(table[b, i // page]) * page + i % page for i in range(n)]
    ts = [None, None]
    if fmt == "nvfp4":
        ts = [(0.0005 + 0.002 * torch.rand(kv_heads, generator=g)) for _ in range(2)]
    c = fp4.KVCache.alloc(fmt, pages, kv_heads, page, dim, "cuda", *(None if t is None else t.cuda() for t in ts))
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
        if t is not None:
            t.view(torch.uint8).fill_(0xFF)
    n = sum(lens)
    k = torch.randn(n, kv_heads, dim, generator=g) * spread
    v = torch.randn(n, kv_heads, dim, generator=g)
    k[:, :, :3] *= 5
    if fmt == "bf16":
        k, v = k.to(torch.bfloat16).float(), v.to(torch.bfloat16).float()
    fp4.kv_cache_append(c, k.cuda(), v.cuda(), torch.tensor(slots, dtype=torch.int64, device="cuda"))
    held = []
    for x, t in ((k, ts[0]), (v, ts[1])):
        if fmt == "bf16":
            held.append(x.double())
        elif n == 0:
            held.append(x.double())
        else:
            t = None if t is None else t.numpy()
            held.append(torch.from_numpy(ref.decode_rows(fmt, *ref.encode_rows(fmt, x.numpy(), t), t)))
    return c, table.cuda(), held[0], held[1]


def _decode_ref(q, k, v, lens, window, scale):
    parts, at = [], 0
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        parts.append(ref.attention(q[b:b + 1].double().cpu(), k[at:at + n], v[at:at + n], scale, [first], [n]))
        at += n
    return [torch.cat(x) for x in zip(*parts)]


def _vsum(v, lens, heads, dim):
    """Per sequence a bound of sum |v| (for the f16 weights' absolute error)."""
    at, rows = 0, []
    for n in lens:
        x = v[at:at + n].abs().sum(0)
        rows.append(x.repeat_interleave(heads // x.shape[0], 0) if n else torch.zeros(heads, dim, dtype=torch.float64))
        at += n
    return torch.stack(rows)


def _check_decode(fmt, lens, heads, kv_heads, dim, page, window=0, seed=0, scale=None, dtype=torch.float32, spread=1.0):
    fp4 = _fp4()
    c, table, k, v = _filled(fp4, fmt, lens, kv_heads, dim, page, seed, spread)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(len(lens), heads, dim, generator=g).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.full((len(lens), heads), 7.0, device="cuda")
    out = fp4.attn_decode_paged(q.cuda(), c, table, n, scale=scale, window=window, dtype=dtype, lse=lse)
    s = dim ** -0.5 if scale is None else scale
    want = _decode_ref(q, k, v, lens, window, s)
    ref.check(out, lse, want, dim, WEIGHT_ULP[fmt], f"decode {fmt} {lens} {heads}/{kv_heads}x{dim} page {page} window {window}",
              _vsum(v, lens, heads, dim) if fmt == "nvfp4" else None)
    return out


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 160, 255, 256, 257]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_lengths(fmt, dim, page):
    _check_decode(fmt, EDGES, 4, 2, dim, page, seed=dim + page)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (7, 1), (10, 2), (16, 1), (17, 1), (40, 2), (32, 32)])
def test_decode_head_layouts(fmt, heads, kv_heads):
    _check_decode(fmt, [70, 5, 0, 200], heads, kv_heads, 128 if heads != 16 else 64, 32, seed=heads)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window", [1, 16, 33, 128, 4096])
def test_decode_window(fmt, window):
    _check_decode(fmt, [0, 1, 40, 129, 300, 511], 8, 2, 64 if window == 33 else 128, 16, window=window, seed=window)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_long_split(fmt):
    """One long sequence beside short ones: its rows are shared by many workgroups and joined."""
    _check_decode(fmt, [3, 20011, 0, 1], 2, 1, 64, 256, seed=5)
    _check_decode(fmt, [4099], 6, 2, 128, 128, seed=6, spread=3.0)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_decode_many_sequences(fmt):
    """More sequences than lanes of a wave, several whole rows per workgroup."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 60, 700)]
    _check_decode(fmt, lens, 2, 1, 64, 16, seed=7)


@pytest.mark.parametrize("scale", [0.0, 0.01, 4.0])
def test_decode_scale(scale):
    _check_decode("bf16", [100, 1, 33], 4, 2, 128, 16, scale=scale, seed=8)
    _check_decode("nvfp4", [100, 1, 33], 4, 2, 128, 16, scale=scale, seed=9)


def test_decode_rising_scores():
    """Scores that grow along the sequence move the running maximum again and again; falling ones never."""
    fp4 = _fp4()
    n, dim = 700, 64
    for sign in (1.0, -1.0):
        k = torch.zeros(n, 1, dim)
        k[:, 0, 0] = sign * torch.arange(n) / 2.0
        v = torch.randn(n, 1, dim, generator=torch.Generator().manual_seed(1))
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        c = fp4.KVCache.alloc("bf16", 11, 1, 64, dim)
        fp4.kv_cache_append(c, k.cuda(), v.cuda(), torch.arange(n, device="cuda"))
        q = torch.zeros(1, 3, dim)
        q[0, :, 0] = torch.tensor([1.0, 8.0, -1.0])
        q = q.to(torch.bfloat16)
        table = torch.arange(11, dtype=torch.int32, device="cuda")[None]
        lse = torch.empty(1, 3, device="cuda")
        out = fp4.attn_decode_paged(q.cuda(), c, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0,
                                    dtype=torch.float32, lse=lse)
        want = ref.attention(q.double(), k.double(), v.double(), 1.0, [0], [n])
        ref.check(out, lse, want, dim, 2.0 ** -8, f"rising {sign}")


def test_decode_output_types_and_strides():
    """bf16 output is the fp32 one rounded; q and out as strided views, a strided block table."""
    fp4 = _fp4()
    lens = [77, 0, 300]
    c, table, _, _ = _filled(fp4, "mxfp8", lens, 2, 128, 16, 11)
    big = torch.randn(3, 20, 128, device="cuda").to(torch.bfloat16)
    q = big[:, 4:12]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = fp4.attn_decode_paged(q, c, table, n, dtype=torch.float32)
    b = fp4.attn_decode_paged(q.contiguous(), c, table, n)
    assert torch.equal(a.to(torch.bfloat16), b)
    hold = torch.full((3, 8, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.cat([table, table], 1)[:, :table.shape[1]]
    fp4.attn_decode_paged(q, c, wide, n, out=hold[:, :, 0])
    assert torch.equal(hold[:, :, 0], b) and bool((hold[:, :, 1] == 9.0).all())
    qt = big.transpose(0, 1)[4:12].transpose(0, 1)  # head stride over sequence stride
    assert torch.equal(fp4.attn_decode_paged(qt, c, table, n), b)


def test_decode_bad_ids_and_lengths_stay_inside():
    """Page ids outside the cache and lengths outside the table are clamped: no access outside the buffers."""
    fp4 = _fp4()
    c, table, _, _ = _filled(fp4, "bf16", [64, 64], 1, 64, 16, 12)
    for t in (c.k_codes, c.v_codes):
        t.fill_(1.0)
    table[0, 1], table[1, 2] = -5, 10 ** 6
    n = torch.tensor([10 ** 9, -3], dtype=torch.int32, device="cuda")
    q = torch.ones(2, 1, 64, device="cuda", dtype=torch.bfloat16)
    out = fp4.attn_decode_paged(q, c, table, n)
    assert bool((out[0] == 1).all()) and bool((out[1] == 0).all())


def test_decode_repeats_streams_graph():
    """The same bits on every call, on another stream, and from a captured graph whose lengths and
    queries change between replays."""
    fp4 = _fp4()
    lens = [900, 5, 0, 333]
    c, table, _, _ = _filled(fp4, "mxfp4", lens, 2, 128, 16, 13)
    q = torch.randn(4, 8, 128, device="cuda").to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = fp4.attn_decode_paged(q, c, table, n)
    assert torch.equal(first, fp4.attn_decode_paged(q, c, table, n))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fp4.attn_decode_paged(q, c, table, n)
    side.synchronize()
    assert torch.equal(first, other)
    ws = fp4.attn_decode_paged_workspace(c, 4, 8, table.shape[1])
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4.attn_decode_paged(q, c, table, n, out=out, workspace=ws)
    for step in range(4):
        q.copy_(torch.randn(4, 8, 128, device="cuda").to(torch.bfloat16))
        n.copy_(torch.tensor([900 - 250 * step, 5 + step, step, 333], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        # (positions that were never written hold NaN: the bits are compared)
        again = fp4.attn_decode_paged(q, c, table, n)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)), step


def test_decode_parts_join_by_lse():
    """Windowed and whole results agree through the logarithms of their sums."""
    fp4 = _fp4()
    c, table, k, v = _filled(fp4, "bf16", [500], 1, 64, 16, 14)
    q = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    lse = [torch.empty(1, 4, device="cuda") for _ in range(3)]
    n = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    whole = fp4.attn_decode_paged(q, c, table, n(500), lse=lse[0], dtype=torch.float32)
    head = fp4.attn_decode_paged(q, c, table, n(380), lse=lse[1], dtype=torch.float32)
    tail = fp4.attn_decode_paged(q, c, table, n(500), window=120, lse=lse[2], dtype=torch.float32)
    assert torch.allclose(torch.logaddexp(lse[1], lse[2]), lse[0], atol=2e-6)
    w = [torch.exp(x - lse[0])[..., None] for x in lse[1:]]
    assert float((w[0] * head + w[1] * tail - whole).abs().max()) < 3 * 2.0 ** -8 * float(v.abs().max())


# ------------------------------------------------------------------ prompts --

def _prompt(lq, lk, heads, kv_heads, dim, causal=True, window=0, scale=None, dtype=torch.float32, seed=0, fused=False):
    fp4 = _fp4()
    g = torch.Generator().manual_seed(seed)
    tq, tk = sum(lq), sum(lk)
    if fused:  # q, k, v as columns of one projection's output
        qkv = torch.randn(tq, heads + 2 * kv_heads, dim, generator=g).to(torch.bfloat16).cuda()
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    else:
        q = torch.randn(tq, heads, dim, generator=g).to(torch.bfloat16).cuda()
        k = torch.randn(tk, kv_heads, dim, generator=g).to(torch.bfloat16).cuda()
        v = torch.randn(tk, kv_heads, dim, generator=g).to(torch.bfloat16).cuda()
    cu = [torch.tensor(np.cumsum([0] + x), dtype=torch.int32, device="cuda") for x in (lq, lk)]
    lse = torch.full((tq, heads), 7.0, device="cuda")
    out = fp4.attn_prefill(q, k, v, *cu, causal=causal, window=window, scale=scale, dtype=dtype, lse=lse)
    parts, a, b = [], 0, 0
    s = dim ** -0.5 if scale is None else scale
    for n, m in zip(lq, lk):
        pos = np.arange(n) + m - n
        last = np.minimum(pos + 1, m) if causal else np.full(n, m)
        first = np.maximum(0, pos - window + 1) if window else np.zeros(n, int)
        parts.append(ref.attention(q[a:a + n].double().cpu(), k[b:b + m].double().cpu(), v[b:b + m].double().cpu(), s, first, last))
        a, b = a + n, b + m
    want = [torch.cat(x) for x in zip(*parts)]
    ref.check(out, lse, want, dim, 2.0 ** -8, f"prompt {lq} {lk} {heads}/{kv_heads}x{dim} causal {causal} window {window}")
    return out


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_lengths(dim, causal):
    lens = [1, 0, 2, 31, 33, 63, 64, 65, 127, 130]
    _prompt(lens, lens, 2, 1, dim, causal, seed=dim)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (5, 1), (6, 2), (16, 1), (21, 3), (40, 8)])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_head_layouts(heads, kv_heads, dim):
    _prompt([40, 3], [40, 3], heads, kv_heads, dim, seed=heads, fused=True)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_longer_and_shorter_keys(dim):
    """Chunks behind a cached context, single queries, and more queries than keys (the first see nothing)."""
    _prompt([1, 5, 70, 20, 9, 4], [300, 133, 71, 0, 4, 64], 4, 2, dim, seed=3)
    _prompt([5, 20, 9], [133, 0, 4], 4, 2, dim, causal=False, seed=4)


@pytest.mark.parametrize("window", [1, 2, 64, 100, 10 ** 6])
def test_prompt_window(window):
    _prompt([150, 1, 40], [150, 200, 260], 4, 2, 64, window=window, seed=window % 97)
    _prompt([90], [130], 2, 1, 128, window=window, seed=window % 89)
    _prompt([70], [100], 2, 1, 256, window=window, causal=False, seed=window % 83)


def test_prompt_many_sequences():
    """More sequences than lanes of a wave; empty ones between."""
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 9, 300)]
    _prompt(lens, lens, 2, 1, 64, seed=9)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_long_rows(dim):
    """Several row tiles and many key tiles, sampled rows."""
    fp4 = _fp4()
    g = torch.Generator().manual_seed(2)
    n, heads, kv = 1500, 6, 2
    q, k, v = (torch.randn(n, h, dim, generator=g).to(torch.bfloat16) for h in (heads, kv, kv))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lse = torch.empty(n, heads, device="cuda")
    out = fp4.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, cu, dtype=torch.float32, lse=lse)
    rows = [0, 1, 63, 64, 500, 777, 1023, 1024, 1498, 1499]
    want = ref.attention(q[rows].double(), k.double(), v.double(), dim ** -0.5, [0] * len(rows), [r + 1 for r in rows])
    ref.check(out[rows], lse[rows], want, dim, 2.0 ** -8, f"long {dim}")


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_few_rows_long_context(dim):
    """A few queries behind long contexts: the keys are split among workgroups and joined.  Contexts
    shorter than a part beside them, a window that leaves parts empty, and one that cuts."""
    for lq, lk, window in (([1], [9000], 0), ([3, 1, 0, 2], [5000, 7, 0, 2049], 0), ([33], [6000], 0),
                           ([5, 4], [4100, 100], 700), ([2], [5000], 1)):
        _prompt(lq, lk, 4, 2, dim, window=window, seed=lk[0])
    _prompt([4], [5000], 4, 2, dim, causal=False, seed=1)


def test_prompt_others_are_not_read():
    """Keys and values of other sequences hold NaN and infinities; keys that are masked may too."""
    fp4 = _fp4()
    lens, dim = [50, 30, 77], 64
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(sum(lens), h, dim, generator=g).to(torch.bfloat16) for h in (4, 2, 2))
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    clean = fp4.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, cu)
    k[50:80], v[50:80] = float("nan"), float("inf")
    k[156, 1] = float("nan")  # seen by the last query of its head only
    out = fp4.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, cu)
    assert torch.equal(out[:50], clean[:50]) and torch.equal(out[80:156], clean[80:156])
    assert torch.equal(out[156, :2], clean[156, :2]) and bool(torch.isnan(out[156, 2:]).all())


def test_prompt_extreme_scores():
    """Scores far apart and of the type's largest values: no overflow where the softmax is defined."""
    fp4 = _fp4()
    dim, n = 64, 130
    q, k, v = torch.zeros(n, 1, dim), torch.zeros(n, 1, dim), torch.randn(n, 1, dim, generator=torch.Generator().manual_seed(5))
    q[:, 0, 0], k[:, 0, 0] = 2.0 ** 60, -(2.0 ** 60)
    k[::7, 0, 0] = 2.0 ** 60
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = fp4.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, cu, dtype=torch.float32, scale=1.0)
    for i in range(n):
        want = v[0:i + 1:7, 0].double().mean(0)
        assert float((out[i, 0].double().cpu() - want).abs().max()) < 2.0 ** -8 * float(v.float().abs().max())


def test_prompt_output_types_strides_streams():
    fp4 = _fp4()
    lens, dim = [70, 33], 128
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(sum(lens), h, dim, generator=g).to(torch.bfloat16).cuda() for h in (6, 2, 2))
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    a = fp4.attn_prefill(q, k, v, cu, cu, dtype=torch.float32)
    b = fp4.attn_prefill(q, k, v, cu, cu)
    assert torch.equal(a.to(torch.bfloat16), b)
    hold = torch.full((103, 6, 2, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    heads_first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    fp4.attn_prefill(*heads_first, cu, cu, out=hold[:, :, 1])
    assert torch.equal(hold[:, :, 1], b) and bool((hold[:, :, 0] == 9.0).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fp4.attn_prefill(q, k, v, cu, cu)
    side.synchronize()
    assert torch.equal(other, b)


def test_prompt_empty():
    fp4 = _fp4()
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert fp4.attn_prefill(e, e, e, z, z).shape == (0, 2, 64)
    q = torch.randn(5, 2, 64, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    for causal in (True, False):
        lse = torch.empty(5, 2, device="cuda")
        out = fp4.attn_prefill(q, e, e, cu, z, causal=causal, lse=lse)
        assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


def test_prompt_then_decode():
    """A prompt goes through the cache: its chunk's attention over what is read back equals, and the next
    token's attention over the cache agrees with the prompt's last row."""
    fp4 = _fp4()
    n, heads, kv, dim, page = 200, 8, 2, 128, 32
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(n, h, dim, generator=g).to(torch.bfloat16).cuda() for h in (heads, kv, kv))
    c = fp4.KVCache.alloc("bf16", 8, kv, page, dim)
    table = torch.tensor([[3, 1, 4, 0, 5, 7, 2, 6]], dtype=torch.int32, device="cuda")
    i = torch.arange(n, device="cuda")
    fp4.kv_cache_append(c, k, v, table[0, i // page].long() * page + i % page)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    whole = fp4.attn_prefill(q, k, v, cu, cu, dtype=torch.float32)
    kr, vr = fp4.kv_cache_read(c, table, cu, n)
    chunk = fp4.attn_prefill(q[120:], kr, vr, torch.tensor([0, 80], dtype=torch.int32, device="cuda"), cu, dtype=torch.float32)
    # both round their weights to bf16 in their own order of tiles
    lim = 2 * 2.0 ** -8 * float(v.float().abs().max())
    assert float((chunk - whole[120:]).abs().max()) < lim
    one = fp4.attn_decode_paged(q[-1:], c, table, torch.tensor([n], dtype=torch.int32, device="cuda"), dtype=torch.float32)
    assert float((one[0] - whole[-1]).abs().max()) < lim
