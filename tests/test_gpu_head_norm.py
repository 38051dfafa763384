"""Norm and rotation of heads on the GPU against the formula in 64 bits, and the form that writes the cache
against the two calls it stands for."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _fp4():
    import block_scaled_fp4_04_amd as fp4

    return fp4


def _ref(x, positions, freqs, weight, eps, interleaved):
    """Rows in float64, and what an error of the pair (a, b) is measured against: |a| + |b|."""
    y = x.double().cpu()
    if eps is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    size = y.abs()
    rot = 0 if freqs is None else 2 * freqs.shape[0]
    if rot:
        a = positions.cpu().double()[:, None] * freqs.cpu()
        c, s = a.cos()[:, None], a.sin()[:, None]
        h = y[..., :rot].clone()
        first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        u, w = h[..., first], h[..., second]
        both = u.abs() + w.abs()
        y, size = y.clone(), size.clone()
        turned = torch.empty_like(h)
        turned[..., first], turned[..., second] = u * c - w * s, w * c + u * s
        y[..., :rot] = turned
        sizes = torch.empty_like(h)
        sizes[..., first] = sizes[..., second] = both
        size[..., :rot] = sizes
    return y, size


def _close(got, ref, what):
    """fp32: a mean of squares has at most 8 + 6 additions and a rounding more (15 2^-24, halved by the root), the
    root and two products 4 2^-24 at most, so 2^-20 covers the norm; cosine and sine are within 2^-22 and the products and
    their sum 2 2^-24 of |a| + |b|.  In all 2^-19.  bf16: half a step, 2^-8, of the result more."""
    y, size = ref
    assert tuple(got.shape) == tuple(y.shape), what
    lim = 2.0 ** -19 * size + (2.0 ** -8 * y.abs() if got.dtype == torch.bfloat16 else 0)
    err = (got.double().cpu() - y).abs()
    bad = ~(err <= lim + 1e-37)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}, worst {float((err / (lim + 1e-37)).max()):.3g}"


def _rows(n, h, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, d, generator=g)
    x[torch.rand(n, h, d, generator=g) < 0.02] *= 50.0
    if n > 1:
        x[1] = 0.0  # a row of zeros stays zeros
        x[0, 0] *= 1e-12
    return x.to(dtype).cuda()


def _weight(shape, seed):
    return (1.0 + 0.3 * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).cuda()


@pytest.mark.parametrize("dim,rot", [(8, 0), (16, 16), (24, 16), (48, 0), (64, 64), (80, 32), (96, 96), (128, 128), (128, 32),
                                     (160, 160), (256, 64), (256, 256), (512, 512), (504, 496)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows(dim, rot, interleaved):
    fp4 = _fp4()
    for n, hq, hk, xt, yt, eps, by_head in [(5, 3, 1, torch.bfloat16, torch.bfloat16, 1e-6, False),
                                            (1, 33, 2, torch.bfloat16, torch.float32, 1e-5, True),
                                            (1100, 5, 3, torch.float32, torch.float32, None, False),
                                            (37, 8, 8, torch.float32, torch.bfloat16, 1e-6, True)]:
        q, k = _rows(n, hq, dim, xt, 1), _rows(n, hk, dim, xt, 2)
        pos = torch.randint(-5, 1 << 20, (n,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
        freqs = fp4.rope_frequencies(rot) if rot else None
        qw, kw = (_weight((h, dim) if by_head else (dim,), h) if eps else None for h in (hq, hk))
        qo, ko = fp4.qk_norm_rope(q, k, pos, freqs, qw, kw, eps=eps, interleaved=interleaved, dtype=yt)
        _close(qo, _ref(q, pos, freqs, qw, eps, interleaved), f"q {n} {hq} {eps} {yt}")
        _close(ko, _ref(k, pos, freqs, kw, eps, interleaved), f"k {n} {hk} {eps} {yt}")


def test_far_positions_and_steep_frequencies():
    fp4 = _fp4()
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 12345678], dtype=torch.int32).cuda()
    freqs = torch.tensor([1.0, 3.14159265358979, 1e-9, 0.5, 2.75, 0.0, 1e-3, 7e-5], dtype=torch.float64).cuda()
    x = _rows(7, 2, 16, torch.float32, 5)
    got, none = fp4.qk_norm_rope(x, None, pos, freqs, dtype=torch.float32)
    assert none is None
    # 64-bit angles of 2^33 radians carry 2^-20 of their own in the reference: take the angle modulo 2 pi from its parts
    y = x.double().cpu()
    import math
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    a = torch.tensor([[float(Fraction(int(p)) * Fraction(float(f)) % (2 * pi)) for f in freqs.cpu()] for p in pos.cpu()], dtype=torch.float64)
    c, s = a.cos()[:, None], a.sin()[:, None]
    u, w = y[..., :8], y[..., 8:]
    want = torch.cat([u * c - w * s, w * c + u * s], -1)
    size = (u.abs() + w.abs()).repeat(1, 1, 2)
    # the product of position and frequency is rounded at 2^-53 of up to 2^33 radians, twice
    err = (got.double().cpu() - want).abs()
    assert bool((err <= (2.0 ** -19 + 2.0 ** -18 * (pos.cpu().double().abs() / 2 ** 31)[:, None, None]) * size + 1e-37).all()), float((err / size.clamp(min=1e-30)).max())
    assert math.isfinite(float(err.max()))


@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_and_in_place(interleaved):
    fp4 = _fp4()
    n, hq, hk, d = 41, 6, 2, 64
    whole = _rows(n, hq + 2 * hk, d, torch.bfloat16, 7)
    q, k = whole[:, :hq], whole[:, hq:hq + hk]
    pos = torch.arange(n, dtype=torch.int32).cuda() * 17
    freqs, qw, kw = fp4.rope_frequencies(d, 5e5), _weight((d,), 1), _weight((hk, d), 2)
    args = (pos, freqs, qw, kw)
    want = fp4.qk_norm_rope(q, k, *args, eps=1e-6, interleaved=interleaved)
    _close(want[0], _ref(q, pos, freqs, qw, 1e-6, interleaved), "columns of a projection")
    # heads outermost, repeated rows, a view with room between the rows
    hf = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(fp4.qk_norm_rope(hf, k, *args, eps=1e-6, interleaved=interleaved)[0], want[0])
    same = k[:, :1].expand(n, hk, d)
    got = fp4.qk_norm_rope(q, same, *args, eps=1e-6, interleaved=interleaved)[1]
    _close(got, _ref(same, pos, freqs, kw, 1e-6, interleaved), "one head repeated")
    room = torch.full((n, hq + 3, d + 32), 7.0, dtype=torch.bfloat16, device="cuda")
    fp4.qk_norm_rope(q, k, *args, eps=1e-6, interleaved=interleaved, q_out=room[:, 2:2 + hq, :d])
    assert torch.equal(room[:, 2:2 + hq, :d], want[0])
    assert bool((room[:, :2] == 7).all()) and bool((room[:, :, d:] == 7).all()) and bool((room[:, 2 + hq:] == 7).all())
    # in place; the values' columns stay
    before = whole.clone()
    got = fp4.qk_norm_rope(q, k, *args, eps=1e-6, interleaved=interleaved, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(whole[:, hq + hk:], before[:, hq + hk:])


def test_nonfinite_rows_stay_apart():
    """A row with an infinity or NaN spoils itself only."""
    fp4 = _fp4()
    for dim in (64, 80, 128):
        x = _rows(9, 5, dim, torch.float32, 11)
        pos = torch.arange(9, dtype=torch.int32).cuda()
        args = (pos, fp4.rope_frequencies(32), _weight((dim,), 1))
        clean = fp4.qk_norm_rope(x, None, *args, eps=1e-6, dtype=torch.float32)[0]
        x[3, 2, 7], x[4, 0, 50] = float("nan"), float("inf")
        got = fp4.qk_norm_rope(x, None, *args, eps=1e-6, dtype=torch.float32)[0]
        hit = torch.zeros(9, 5, dtype=torch.bool)
        hit[3, 2] = hit[4, 0] = True
        assert torch.equal(got[~hit.cuda()], clean[~hit.cuda()])
        assert bool(got[3, 2].isnan().all())
        # not normed: values that do not turn with it are untouched
        got = fp4.qk_norm_rope(x, None, pos, fp4.rope_frequencies(32), dtype=torch.float32)[0]
        assert torch.equal(got[4, 0, 32:], x[4, 0, 32:]) and bool(got[3, 2, [8, 9, 40]].isfinite().all())


def test_many_tokens():
    """More tokens than one wave each: the first, the last and those between give what they give alone."""
    fp4 = _fp4()
    n, d = 70001, 64
    q = torch.randn(n, 2, d, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    freqs, w = fp4.rope_frequencies(d), _weight((d,), 4)
    got = fp4.qk_norm_rope(q, None, pos, freqs, w, eps=1e-6)[0]
    at = torch.tensor([0, 1, 255, 256, 4095, 4096, 65535, 65536, n - 1], device="cuda")
    alone = fp4.qk_norm_rope(q[at], None, pos[at], freqs, w, eps=1e-6)[0]
    assert torch.equal(got[at], alone)
    _close(alone, _ref(q[at], pos[at], freqs, w, 1e-6, False), "tokens picked")


def test_past_4gib():
    """Offsets past 32 bits: rows of a buffer of 6 GB."""
    fp4 = _fp4()
    n, step = 4, 3 * (1 << 28)  # elements between tokens
    base = torch.empty(n * step, dtype=torch.bfloat16, device="cuda")
    q = base.as_strided((n, 3, 128), (step, 128, 1))
    q.copy_(_rows(n, 3, 128, torch.bfloat16, 9))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    want = fp4.qk_norm_rope(q.contiguous(), None, pos, fp4.rope_frequencies(128))[0]
    assert torch.equal(fp4.qk_norm_rope(q, None, pos, fp4.rope_frequencies(128))[0], want)
    fp4.qk_norm_rope(q, None, pos, fp4.rope_frequencies(128), q_out=q)
    assert torch.equal(q, want)


def _cache(fp4, fmt, pages, heads, page, dim):
    ts = [None, None]
    if fmt == "nvfp4":
        ts = [(0.001 + 0.01 * torch.rand(heads, generator=torch.Generator().manual_seed(s))).cuda() for s in (1, 2)]
    c = fp4.KVCache.alloc(fmt, pages, heads, page, dim, "cuda", *ts)
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
        if t is not None:
            t.view(torch.uint8).fill_(0xA5)  # what is not written has to stay
    return c


def _same(a, b):
    for x in ("k_codes", "v_codes", "k_scales", "v_scales"):
        u, w = getattr(a, x), getattr(b, x)
        if u is not None:
            assert torch.equal(u.view(torch.uint8), w.view(torch.uint8)), x


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("dim,heads,kv,page", [(64, 4, 1, 16), (128, 15, 5, 64), (256, 2, 2, 256)])
def test_append_is_the_two_calls(fmt, dim, heads, kv, page):
    """Keys quantized from fp32 are what kv_cache_append makes of fp32 rows; q is what qk_norm_rope gives."""
    fp4 = _fp4()
    for n, xt, rule, eps, inter, rot in [(37, torch.bfloat16, "ocp", 1e-6, False, dim), (1, torch.float32, "ceil", None, True, 32),
                                         (1200, torch.bfloat16, "ceil", 1e-6, True, 0)]:
        pages = (n + page - 1) // page + 3
        whole = _rows(n, heads + 2 * kv, dim, xt, 3)
        q, k, v = whole.split([heads, kv, kv], 1)
        g = torch.Generator().manual_seed(5)
        slots = torch.randperm(pages * page, generator=g)[:n]
        if n > 5:
            slots[2], slots[5] = -1, pages * page  # skipped
        slots = slots.cuda()
        pos = torch.randint(0, 100000, (n,), generator=g, dtype=torch.int32).cuda()
        freqs = fp4.rope_frequencies(rot) if rot else None
        qw, kw = (_weight((h, dim), h) if eps else None for h in (heads, kv))
        one, two = _cache(fp4, fmt, pages, kv, page, dim), _cache(fp4, fmt, pages, kv, page, dim)
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = fp4.qk_norm_rope_append(one, q, k, v, pos, slots, freqs, qw, kw, eps=eps, interleaved=inter, rule=rule, nonfinite=bad)
        want, kr = fp4.qk_norm_rope(q, k, pos, freqs, qw, kw, eps=eps, interleaved=inter, dtype=torch.float32)
        fp4.kv_cache_append(two, kr, v.float(), slots, rule=rule)
        assert torch.equal(got, want.to(torch.bfloat16))
        _same(one, two)
        assert int(bad) == 0
        if xt == torch.bfloat16:  # q in place
            again, three = whole.clone(), _cache(fp4, fmt, pages, kv, page, dim)
            qq, kk, vv = again.split([heads, kv, kv], 1)
            fp4.qk_norm_rope_append(three, qq, kk, vv, pos, slots, freqs, qw, kw, eps=eps, interleaved=inter, rule=rule, q_out=qq)
            assert torch.equal(qq, got) and torch.equal(again[:, heads:], whole[:, heads:])
            _same(three, two)
        if n > 5 and fmt != "bf16":
            v = v.clone()
            v[2, 0, 0] = float("nan")  # a token that is not stored
            fp4.qk_norm_rope_append(one, q, k, v, pos, slots, freqs, qw, kw, eps=eps, interleaved=inter, rule=rule, nonfinite=bad)
            assert int(bad) == 0
            v[3, 0, 0] = float("nan")
            fp4.qk_norm_rope_append(one, q, k, v, pos, slots, freqs, qw, kw, eps=eps, interleaved=inter, rule=rule, nonfinite=bad)
            assert int(bad) == 1


def test_no_tokens():
    fp4 = _fp4()
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    a, b = fp4.qk_norm_rope(q, q, pos, fp4.rope_frequencies(64))
    assert a.shape == b.shape == (0, 4, 64)


def test_captured_and_on_another_stream():
    fp4 = _fp4()
    n, heads, kv, dim, page = 16, 8, 2, 128, 16
    side = torch.cuda.Stream()
    cache, want = _cache(fp4, "mxfp8", 4, kv, page, dim), _cache(fp4, "mxfp8", 4, kv, page, dim)
    whole = _rows(n, heads + 2 * kv, dim, torch.bfloat16, 3)
    q, k, v = whole.split([heads, kv, kv], 1)
    pos, slots = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n,), -1, dtype=torch.int64, device="cuda")
    freqs, w = fp4.rope_frequencies(dim), _weight((dim,), 1)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp4.qk_norm_rope_append(cache, q, k, v, pos, slots, freqs, w, w, eps=1e-6)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = fp4.qk_norm_rope_append(cache, q, k, v, pos, slots, freqs, w, w, eps=1e-6)
        for i in range(3):
            whole.copy_(_rows(n, heads + 2 * kv, dim, torch.bfloat16, 20 + i))
            pos.fill_(100 * i)
            slots.copy_(torch.randperm(4 * page)[:n])
            graph.replay()
            got = fp4.qk_norm_rope_append(want, q, k, v, pos, slots, freqs, w, w, eps=1e-6)
            side.synchronize()
            assert torch.equal(out, got)
            _same(cache, want)


def test_cache_past_4gib():
    """Pages whose codes lie past 4 GiB of the cache."""
    fp4 = _fp4()
    kv, page, dim, pages = 2, 128, 128, 70000
    cache = fp4.KVCache.alloc("bf16", pages, kv, page, dim)
    n = 5
    whole = _rows(n, 4 + 2 * kv, dim, torch.bfloat16, 3)
    q, k, v = whole.split([4, kv, kv], 1)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") + 100
    slots = torch.tensor([0, pages * page - 1, 66000 * page + 7, -1, 33000 * page], device="cuda")
    freqs = fp4.rope_frequencies(dim)
    fp4.qk_norm_rope_append(cache, q, k, v, pos, slots, freqs)
    want = fp4.qk_norm_rope(q, k, pos, freqs)[1]
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            assert torch.equal(cache.k_codes[s // page, :, s % page], want[i])
            assert torch.equal(cache.v_codes[s // page, :, s % page], v[i])
    copies = torch.tensor([[66000, 69998, 8], [pages - 1, 1, page]], dtype=torch.int32, device="cuda")
    fp4.kv_cache_copy(cache, copies)
    assert torch.equal(cache.k_codes[69998, :, 7], want[2]) and torch.equal(cache.v_codes[1, :, page - 1], v[1])


def test_recorded_calls():
    """prepare() replays both forms on the same memory."""
    fp4 = _fp4()
    whole = _rows(3, 8, 64, torch.bfloat16, 1)
    q, k, v = whole.split([4, 2, 2], 1)
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    cache = _cache(fp4, "mxfp8", 2, 2, 16, 64)
    slots = torch.arange(3, device="cuda")
    freqs, w = fp4.rope_frequencies(64), _weight((64,), 2)
    outs = []
    call = fp4.prepare(lambda: outs.extend((*fp4.qk_norm_rope(q, k, pos, freqs, w, w, eps=1e-6),
                                            fp4.qk_norm_rope_append(cache, q, k, v, pos, slots, freqs, w, w, eps=1e-6))))
    whole.copy_(_rows(3, 8, 64, torch.bfloat16, 9))
    call()
    want = fp4.qk_norm_rope(q, k, pos, freqs, w, w, eps=1e-6)
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(outs[2], want[0])
    other = _cache(fp4, "mxfp8", 2, 2, 16, 64)
    fp4.qk_norm_rope_append(other, q, k, v, pos, slots, freqs, w, w, eps=1e-6)
    _same(cache, other)


@pytest.mark.parametrize("dtype,dim,rot", [(torch.bfloat16, 128, 128), (torch.float32, 80, 32), (torch.bfloat16, 64, 64)])
def test_rows_past_the_caches(dtype, dim, rot):
    """Over 96 MB of rows: every token is what it is in a small call."""
    fp4 = _fp4()
    heads, kv = 12, 4
    n = (110 << 20) // ((heads + kv) * dim * dtype.itemsize)
    whole = torch.randn(n, heads + kv, dim, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(dtype)
    q, k = whole.split([heads, kv], 1)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 3
    freqs, w = fp4.rope_frequencies(rot), _weight((dim,), 4)
    got = fp4.qk_norm_rope(q, k, pos, freqs, w, w, eps=1e-6, dtype=dtype)
    for at in range(0, n, 9973):
        s = slice(at, at + 1111)
        alone = fp4.qk_norm_rope(q[s], k[s], pos[s], freqs, w, w, eps=1e-6, dtype=dtype)
        assert torch.equal(got[0][s], alone[0]) and torch.equal(got[1][s], alone[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (64, 64, False), (80, 32, True), (512, 0, False), (8, 0, False)])
def test_rows_whose_squares_pass_fp32(dim, rot, interleaved, dtype):
    """Finite rows of any size are normed: values past 10^18, whose squares (or their sum) have no place in fp32, up to the type's largest, beside
    ordinary rows of the same wave."""
    fp4 = _fp4()
    n, h = 23, 5
    x = torch.randn(n, h, dim, generator=torch.Generator().manual_seed(dim))
    for i, size in enumerate((1e15, 1e18, 4e18, 2e19, 1e25, 1e37)):
        x[i, ::2] *= size
    x[7, 1] = 1e-3
    x[7, 1, 3] = -3e38
    x[8, 4] = torch.finfo(dtype).max
    x[8, 4, ::3] *= -1
    x = x.to(dtype).cuda()
    pos = torch.arange(n, dtype=torch.int32).cuda() * 31
    freqs, w = (fp4.rope_frequencies(rot) if rot else None), _weight((h, dim), 1)
    for eps in (1e-30, 1e-6, 1e30):
        got = fp4.qk_norm_rope(x, x[:, 1:4], pos, freqs, w, w[1:4].contiguous(), eps=eps, interleaved=interleaved, dtype=torch.float32)
        want = _ref(x, pos, freqs, w, eps, interleaved)
        _close(got[0], want, f"q {eps}")
        _close(got[1], [t[:, 1:4] for t in want], f"k {eps}")
    if dim >= 64 and dim != 80 and dim != 512:  # the cache write's keys, rounded once
        cache = fp4.KVCache.alloc("bf16", 2, h, 16, dim, "cuda")
        args = (pos, torch.arange(n).cuda(), freqs, w, w)
        q = fp4.qk_norm_rope_append(cache, x, x, x, *args, eps=1e-6, interleaved=interleaved)
        same = fp4.qk_norm_rope(x, x, pos, freqs, w, w, eps=1e-6, interleaved=interleaved)
        assert torch.equal(q, same[0])
        assert torch.equal(cache.k_codes.transpose(1, 2).reshape(32, h, dim)[:n].view(torch.bfloat16), same[1])
