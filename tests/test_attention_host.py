"""What the cache and attention entry points refuse (CPU only; nothing is launched): status codes of
the C ABI, and the binding's own checks of tensors."""
import ctypes
import os

import pytest
import torch

OK, NULL, SHAPE, LAYOUT, DTYPE, WORKSPACE, NO_DEVICE, UNSUPPORTED, HIP = range(9)
FAKE = 1 << 20  # a 16-byte-aligned non-null address; never dereferenced on the host
GPU = torch.cuda.is_available()


@pytest.fixture(scope="module")
def fp4():
    import block_scaled_fp4_04_amd as m

    if not os.path.exists(m.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    m.lib()
    return m


def _cache(fp4, **kw):
    f = dict(format=2, pages=10, kv_heads=2, page_size=16, head_dim=64, k_codes=FAKE, v_codes=FAKE, k_scales=FAKE,
             v_scales=FAKE, k_tscale=FAKE, v_tscale=FAKE)
    f.update(kw)
    c = fp4._KvCacheArg(*f.values())
    return ctypes.byref(c)


CACHE_FAULTS = [(dict(format=4), DTYPE), (dict(format=-1), DTYPE), (dict(pages=0), SHAPE), (dict(kv_heads=0), SHAPE),
                (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=512), SHAPE),
                (dict(head_dim=96), SHAPE), (dict(head_dim=32), SHAPE), (dict(pages=1 << 27), SHAPE),
                (dict(k_codes=None), NULL), (dict(v_codes=FAKE + 8), LAYOUT), (dict(k_scales=None), NULL),
                (dict(v_scales=FAKE + 4), LAYOUT), (dict(k_tscale=None), NULL), (dict(v_tscale=None), NULL)]


def _append(fp4, cache=None, **kw):
    a = dict(cache=_cache(fp4) if cache is None else cache, k=FAKE, v=FAKE, xt=1, tokens=5, kt=128, kh=64, vt=128, vh=64, slots=FAKE,
             rule=0, nonfinite=None, stream=None)
    a.update(kw)
    return fp4.lib().kv_cache_append(*a.values())


def _read(fp4, cache=None, **kw):
    a = dict(cache=_cache(fp4) if cache is None else cache, table=FAKE, seqs=3, width=4, stride=4, cu=FAKE, tokens=50, k=FAKE, v=FAKE,
             yt=1, kt=128, kh=64, vt=128, vh=64, stream=None)
    a.update(kw)
    return fp4.lib().kv_cache_read(*a.values())


def _decode(fp4, cache=None, **kw):
    a = dict(q=FAKE, seqs=3, heads=4, qs=256, qh=64, cache=_cache(fp4) if cache is None else cache, table=FAKE, width=4, stride=4,
             lens=FAKE, scale=0.125, window=0, out=FAKE, ot=1, os=256, oh=64, lse=None, ws=FAKE, wsb=1 << 40,
             stream=None)
    a.update(kw)
    return fp4.lib().attn_decode_paged(*a.values())


def _prefill(fp4, **kw):
    a = dict(q=FAKE, qn=50, heads=4, qt=256, qh=64, k=FAKE, v=FAKE, kn=60, kv=2, dim=64, kt=128, kh=64, vt=128, vh=64,
             cuq=FAKE, cuk=FAKE, seqs=2, scale=0.125, causal=1, window=0, out=FAKE, ot=1, ott=256, oh=64, lse=None,
             ws=None, wsb=0, stream=None)
    a.update(kw)
    return fp4.lib().attn_prefill(*a.values())


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_descriptor(fp4, fault, status):
    for call in (_append, _read, _decode):
        assert call(fp4, _cache(fp4, **fault)) == status
    assert _append(fp4, cache=ctypes.POINTER(fp4._KvCacheArg)()) == NULL


def test_formats_need_only_their_parts(fp4):
    bare = dict(k_scales=None, v_scales=None, k_tscale=None, v_tscale=None)
    want = None if GPU else NO_DEVICE
    for fmt, kw in ((0, bare), (1, dict(k_tscale=None, v_tscale=None)), (3, dict(k_tscale=None, v_tscale=None))):
        if not GPU:
            assert _append(fp4, _cache(fp4, format=fmt, **kw)) == want


def test_append(fp4):
    assert _append(fp4, xt=2) == DTYPE and _append(fp4, rule=2) == DTYPE
    assert _append(fp4, tokens=-1) == SHAPE and _append(fp4, tokens=1 << 40) == SHAPE
    assert _append(fp4, tokens=(1 << 31) // (2 * 2 * 8)) == SHAPE  # 2^31 units of 8 values
    assert _append(fp4, k=None) == NULL and _append(fp4, v=None) == NULL and _append(fp4, slots=None) == NULL
    assert _append(fp4, k=FAKE + 2) == LAYOUT and _append(fp4, kt=-128) == LAYOUT
    assert _append(fp4, kh=68) == LAYOUT and _append(fp4, xt=0, vh=66) == LAYOUT
    assert _append(fp4, tokens=0, k=None, v=None, slots=None) == OK
    if not GPU:
        assert _append(fp4) == NO_DEVICE and _append(fp4, kt=0, kh=0) == NO_DEVICE


def test_read(fp4):
    assert _read(fp4, yt=3) == DTYPE
    assert _read(fp4, seqs=0) == SHAPE and _read(fp4, width=0) == SHAPE and _read(fp4, width=1 << 27) == SHAPE
    assert _read(fp4, tokens=-1) == SHAPE
    assert _read(fp4, table=None) == NULL and _read(fp4, cu=None) == NULL and _read(fp4, k=None) == NULL
    assert _read(fp4, stride=3) == LAYOUT and _read(fp4, kt=32) == LAYOUT and _read(fp4, vh=0) == LAYOUT
    assert _read(fp4, tokens=0, k=None, v=None) == OK
    if not GPU:
        assert _read(fp4) == NO_DEVICE and _read(fp4, seqs=1, stride=0) == NO_DEVICE


def test_decode(fp4):
    assert _decode(fp4, ot=2) == DTYPE
    for bad in (dict(heads=5), dict(heads=0), dict(seqs=0), dict(window=-1), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(width=0), dict(seqs=1 << 23, width=1 << 20, stride=1 << 20)):
        assert _decode(fp4, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(table=None), dict(lens=None), dict(out=None)):
        assert _decode(fp4, **bad) == NULL, bad
    for bad in (dict(q=FAKE + 4), dict(qs=100), dict(oh=32), dict(stride=2), dict(out=FAKE + 8)):
        assert _decode(fp4, **bad) == LAYOUT, bad
    L = fp4.lib()
    need = L.attn_decode_paged_workspace(3, 4, _cache(fp4), 400)
    assert need > 0
    assert L.attn_decode_paged_workspace(0, 4, _cache(fp4), 4) == 0
    assert L.attn_decode_paged_workspace(3, 5, _cache(fp4), 4) == 0
    if not GPU:
        assert _decode(fp4) == NO_DEVICE


def test_prefill(fp4):
    assert _prefill(fp4, ot=2) == DTYPE and _prefill(fp4, causal=2) == DTYPE
    for bad in (dict(heads=5), dict(kv=0), dict(dim=96), dict(qn=-1), dict(kn=-1), dict(kn=1 << 31), dict(qn=1 << 30),
                dict(seqs=0), dict(window=-2), dict(scale=-0.5)):
        assert _prefill(fp4, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(cuq=None), dict(cuk=None), dict(out=None)):
        assert _prefill(fp4, **bad) == NULL, bad
    for bad in (dict(q=FAKE + 2), dict(kt=100), dict(vh=-64), dict(ott=32), dict(out=FAKE + 8)):
        assert _prefill(fp4, **bad) == LAYOUT, bad
    assert _prefill(fp4, qn=0, q=None, k=None, v=None, out=None) == OK
    L = fp4.lib()
    assert L.attn_prefill_workspace(8192, 8, 8192, 2, 64, 1) == 0          # the rows alone fill the chip
    assert L.attn_prefill_workspace(5, 8, 100, 2, 64, 1) == 0              # few keys
    assert L.attn_prefill_workspace(5, 8, 100000, 2, 64, 1) > 0
    assert L.attn_prefill_workspace(5, 9, 100000, 2, 64, 1) == 0
    if not GPU:
        assert _prefill(fp4) == NO_DEVICE and _prefill(fp4, kn=0, k=None, v=None) == NO_DEVICE


def test_binding_refuses(fp4):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        fp4.KVCache("int4", u8(2, 2, 16, 32), u8(2, 2, 16, 32))
    with pytest.raises(ValueError):
        fp4.KVCache("mxfp4", u8(2, 2, 16, 32), u8(2, 2, 16, 32))              # no scales
    with pytest.raises(ValueError):
        fp4.KVCache("mxfp4", u8(2, 2, 16, 32), u8(2, 2, 16, 32), u8(2, 2, 4, 16), u8(2, 2, 4, 16))  # 2 blocks of 32
    with pytest.raises(ValueError):
        fp4.KVCache("mxfp8", u8(2, 2, 16, 96), u8(2, 2, 16, 96))              # head_dim
    with pytest.raises(ValueError):
        fp4.KVCache("mxfp8", u8(2, 2, 24, 64), u8(2, 2, 24, 64))              # page size
    with pytest.raises(TypeError):
        fp4.KVCache("bf16", torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64))
    with pytest.raises(ValueError):
        fp4.KVCache("bf16", bf(2, 2, 16, 64), bf(3, 2, 16, 64))
    with pytest.raises(ValueError):
        fp4.KVCache("bf16", bf(2, 2, 16, 64), bf(2, 2, 16, 64), u8(2, 2, 2, 16))
    with pytest.raises(ValueError):
        fp4.KVCache("nvfp4", u8(2, 2, 16, 32), u8(2, 2, 16, 32), u8(2, 2, 4, 16), u8(2, 2, 4, 16))  # no tscale
    with pytest.raises(ValueError, match="device"):
        fp4.KVCache("bf16", bf(2, 2, 16, 64), bf(2, 2, 16, 64))
    q, k, cu = bf(8, 4, 64), bf(8, 2, 64), i32(3)
    for bad, err in ((dict(q=q.float()), TypeError), (dict(k=bf(8, 3, 64), v=bf(8, 3, 64)), ValueError),
                     (dict(v=bf(9, 2, 64)), ValueError), (dict(k=bf(8, 2, 128), v=bf(8, 2, 128)), ValueError),
                     (dict(cu_seqlens_k=i32(4)), ValueError), (dict(cu_seqlens_q=cu.long()), TypeError),
                     (dict(q=bf(8, 4, 128)[:, :, ::2]), ValueError), (dict(out=bf(8, 4, 128)), ValueError),
                     (dict(lse=torch.zeros(4, 8)), ValueError), (dict(dtype=torch.float16), TypeError),
                     (dict(q=bf(8, 256)), ValueError), (dict(), ValueError)):  # the last: host tensors
        a = dict(q=q, k=k, v=k, cu_seqlens_q=cu, cu_seqlens_k=cu)
        a.update(bad)
        with pytest.raises(err):
            fp4.attn_prefill(**a)
