"""What the calls around the attention refuse (CPU only; nothing is launched): status codes of the C
ABI, and the binding's own checks of tensors."""
import ctypes

import pytest
import torch

from test_attention_host import (CACHE_FAULTS, DTYPE, FAKE, GPU, LAYOUT, NO_DEVICE, NULL, OK, SHAPE, WORKSPACE,  # noqa: F401
                                 _cache, fp4)


def _norm(fp4, **kw):
    a = dict(q=FAKE, k=FAKE, xt=1, tokens=5, heads=4, kv=2, dim=64, qt=256, qh=64, kt=128, kh=64, qw=FAKE, kw=FAKE, qws=0,
             kws=64, eps=1e-6, pos=FAKE, freqs=FAKE, rot=64, inter=0, qo=FAKE, ko=FAKE, yt=1, qot=256, qoh=64, kot=128, koh=64,
             stream=None)
    a.update(kw)
    return fp4.lib().qk_norm_rope(*a.values())


def _norm_append(fp4, cache=None, **kw):
    a = dict(cache=_cache(fp4) if cache is None else cache, q=FAKE, k=FAKE, v=FAKE, xt=1, tokens=5, heads=4, qt=256, qh=64,
             kt=128, kh=64, vt=128, vh=64, qw=FAKE, kw=FAKE, qws=0, kws=64, eps=1e-6, pos=FAKE, freqs=FAKE, rot=64, inter=0,
             slots=FAKE, rule=0, nonfinite=None, qo=FAKE, yt=1, qot=256, qoh=64, stream=None)
    a.update(kw)
    return fp4.lib().qk_norm_rope_append(*a.values())


def _pool(fp4, **kw):
    a = dict(free_list=FAKE, state=FAKE, pages=100, page_size=16)
    a.update(kw)
    return ctypes.byref(fp4._KvPagesArg(*a.values()))


def _extend(fp4, pool=None, **kw):
    a = dict(pool=_pool(fp4) if pool is None else pool, table=FAKE, seqs=3, width=4, stride=4, lens=FAKE, new=FAKE, tokens=9,
             lo=FAKE, so=FAKE, slots=FAKE, pos=FAKE, cuq=None, cuk=None, ws=None, wsb=0, stream=None)
    a.update(kw)
    return fp4.lib().kv_pages_extend(*a.values())


def _collect(fp4, pool=None, **kw):
    a = dict(pool=_pool(fp4) if pool is None else pool, table=FAKE, seqs=3, width=4, stride=4, lens=FAKE, ws=None, wsb=0,
             stream=None)
    a.update(kw)
    return fp4.lib().kv_pages_collect(*a.values())


def _reorder(fp4, **kw):
    a = dict(table=FAKE, batch=3, beams=4, width=5, stride=5, lens=FAKE, parents=FAKE, page=16, out=FAKE, ostride=5,
             copies=FAKE, stream=None)
    a.update(kw)
    return fp4.lib().kv_pages_reorder(*a.values())


def _select(fp4, **kw):
    a = dict(logits=FAKE, xt=1, batch=2, beams=3, vocab=1000, ld=1000, scores=FAKE, done=None, end=0, k=3, so=FAKE, po=FAKE,
             to=FAKE, ws=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    return fp4.lib().beam_select(*a.values())


def test_norm(fp4):
    for bad in (dict(xt=2), dict(yt=-1), dict(inter=2)):
        assert _norm(fp4, **bad) == DTYPE, bad
    for bad in (dict(tokens=-1), dict(tokens=1 << 31), dict(heads=0), dict(heads=65536), dict(kv=-1), dict(dim=60), dict(dim=520),
                dict(dim=0), dict(rot=8), dict(rot=80), dict(rot=-16), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(eps=1e-31)):
        assert _norm(fp4, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(k=None), dict(qw=None), dict(kw=None), dict(pos=None), dict(freqs=None), dict(qo=None),
                dict(ko=None)):
        assert _norm(fp4, **bad) == NULL, bad
    for bad in (dict(q=FAKE + 2), dict(kt=68), dict(qh=-64), dict(qws=2), dict(kws=-64), dict(qw=FAKE + 8), dict(freqs=FAKE + 4),
                dict(qot=32), dict(koh=0), dict(ko=FAKE + 8), dict(xt=0, kt=130)):
        assert _norm(fp4, **bad) == LAYOUT, bad
    assert _norm(fp4, tokens=0, q=None, qo=None) == OK
    if not GPU:
        for fine in (dict(), dict(kv=0, k=None, ko=None, kw=None), dict(eps=0.0, qw=None, kw=None),
                     dict(rot=0, pos=None, freqs=None), dict(qt=0, kh=0)):
            assert _norm(fp4, **fine) == NO_DEVICE, fine


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_descriptor(fp4, fault, status):
    assert _norm_append(fp4, _cache(fp4, **fault)) == status
    assert fp4.lib().kv_cache_copy(_cache(fp4, **fault), FAKE, 3, None) == status


def test_norm_append(fp4):
    for bad in (dict(xt=2), dict(yt=3), dict(inter=-1), dict(rule=2)):
        assert _norm_append(fp4, **bad) == DTYPE, bad
    for bad in (dict(tokens=-1), dict(heads=0), dict(rot=24), dict(rot=128), dict(eps=-1e-6)):
        assert _norm_append(fp4, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(qw=None), dict(kw=None), dict(pos=None), dict(freqs=None),
                dict(slots=None), dict(qo=None)):
        assert _norm_append(fp4, **bad) == NULL, bad
    for bad in (dict(v=FAKE + 4), dict(vt=100), dict(qoh=32), dict(kws=1)):
        assert _norm_append(fp4, **bad) == LAYOUT, bad
    assert _norm_append(fp4, tokens=0, q=None) == OK
    if not GPU:
        assert _norm_append(fp4) == NO_DEVICE
        assert _norm_append(fp4, eps=0.0, qw=None, kw=None, rot=0, pos=None, freqs=None) == NO_DEVICE


POOL_FAULTS = [(dict(pages=0), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=512), SHAPE),
               (dict(pages=1 << 27), SHAPE), (dict(free_list=None), NULL), (dict(state=None), NULL)]


@pytest.mark.parametrize("fault,status", POOL_FAULTS)
def test_pool_descriptor(fp4, fault, status):
    for call in (_extend, _collect):
        assert call(fp4, _pool(fp4, **fault)) == status
        assert call(fp4, ctypes.POINTER(fp4._KvPagesArg)()) == NULL


def test_pages(fp4):
    L = fp4.lib()
    for call in (_extend, _collect):
        for bad in (dict(seqs=0), dict(seqs=1 << 24), dict(width=0), dict(width=1 << 26)):
            assert call(fp4, **bad) == SHAPE, bad
        for bad in (dict(table=None), dict(lens=None)):
            assert call(fp4, **bad) == NULL, bad
        assert call(fp4, stride=3) == LAYOUT
        if not GPU:
            assert call(fp4) == NO_DEVICE and call(fp4, seqs=1, stride=0) == NO_DEVICE
    assert _extend(fp4, tokens=-1) == SHAPE and _extend(fp4, tokens=1 << 30) == SHAPE
    for bad in (dict(new=None), dict(lo=None), dict(so=None), dict(slots=None), dict(pos=None)):
        assert _extend(fp4, **bad) == NULL, bad
    if not GPU:
        assert _extend(fp4, tokens=0, slots=None, pos=None) == NO_DEVICE
    need = L.kv_pages_extend_workspace(3000, 5)
    assert need > 0 and L.kv_pages_extend_workspace(3, 1 << 20) > 0 and L.kv_pages_extend_workspace(64, 64) == 0
    assert _extend(fp4, seqs=3000, tokens=5) == WORKSPACE
    assert _extend(fp4, seqs=3000, tokens=5, ws=FAKE, wsb=need - 1) == WORKSPACE
    assert _extend(fp4, seqs=3000, tokens=5, ws=FAKE + 4, wsb=need) == WORKSPACE
    need = L.kv_pages_collect_workspace(1 << 20, 3, 4)
    assert need > 0 and L.kv_pages_collect_workspace(100, 3, 4) == 0 and L.kv_pages_collect_workspace(0, 3, 4) == 0
    assert _collect(fp4, _pool(fp4, pages=1 << 20)) == WORKSPACE


def test_reorder_and_copy(fp4):
    for bad in (dict(batch=0), dict(beams=0), dict(beams=65), dict(page=8), dict(page=33), dict(width=0), dict(batch=1 << 24),
                dict(batch=1 << 22, beams=4), dict(batch=1 << 18, beams=1, width=1 << 14, stride=1 << 14, ostride=1 << 14)):
        assert _reorder(fp4, **bad) == SHAPE, bad
    for bad in (dict(table=None), dict(lens=None), dict(parents=None), dict(out=None), dict(copies=None)):
        assert _reorder(fp4, **bad) == NULL, bad
    for bad in (dict(stride=4), dict(out=FAKE + 64, ostride=4), dict(ostride=6)):  # the last: in place at another stride
        assert _reorder(fp4, **bad) == LAYOUT, bad
    L = fp4.lib()
    assert L.kv_cache_copy(_cache(fp4), FAKE, -1, None) == SHAPE and L.kv_cache_copy(_cache(fp4), FAKE, 1 << 22, None) == SHAPE
    assert L.kv_cache_copy(_cache(fp4), None, 3, None) == NULL and L.kv_cache_copy(_cache(fp4), None, 0, None) == OK
    if not GPU:
        assert _reorder(fp4) == NO_DEVICE and L.kv_cache_copy(_cache(fp4), FAKE, 3, None) == NO_DEVICE


def test_select(fp4):
    assert _select(fp4, xt=2) == DTYPE
    for bad in (dict(batch=0), dict(beams=0), dict(beams=65), dict(vocab=0), dict(vocab=1 << 30, ld=1 << 30), dict(k=0), dict(k=65), dict(vocab=1, ld=1, k=4),
                dict(end=-1), dict(end=1000), dict(batch=1 << 21), dict(batch=1 << 20, beams=16, vocab=5, ld=5)):
        assert _select(fp4, **bad) == SHAPE, bad
    for bad in (dict(logits=None), dict(scores=None), dict(so=None), dict(po=None), dict(to=None)):
        assert _select(fp4, **bad) == NULL, bad
    assert _select(fp4, ld=999) == LAYOUT and _select(fp4, logits=FAKE + 1) == LAYOUT and _select(fp4, xt=0, logits=FAKE + 2) == LAYOUT
    L = fp4.lib()
    need = L.beam_select_workspace(2, 3, 1000, 3, 1)
    assert need > 0 and L.beam_select_workspace(2, 3, 1000, 65, 1) == 0 and L.beam_select_workspace(2, 3, 1000, 3, 5) == 0
    assert _select(fp4, wsb=need - 1) == WORKSPACE and _select(fp4, ws=None) == WORKSPACE and _select(fp4, ws=FAKE + 8) == WORKSPACE
    if not GPU:
        assert _select(fp4, wsb=need) == NO_DEVICE and _select(fp4, logits=FAKE + 2, ld=1001) == NO_DEVICE


def _i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def test_binding_refuses_norms(fp4):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    q, k, w = bf(8, 4, 64), bf(8, 2, 64), torch.ones(64)
    freqs = fp4.rope_frequencies(64, device="cpu")
    assert freqs.dtype == torch.float64 and freqs.shape == (32,) and float(freqs[0]) == 1.0
    good = dict(q=q, k=k, positions=_i32(8), freqs=freqs, q_weight=w, k_weight=torch.ones(2, 64), eps=1e-6)
    for bad, err in ((dict(q=q.half()), TypeError), (dict(k=k.float()), ValueError), (dict(k=bf(9, 2, 64)), ValueError),
                     (dict(k=bf(8, 2, 128)), ValueError), (dict(k=bf(8, 0, 64)), ValueError), (dict(eps=0.0), ValueError),
                     (dict(eps=None), ValueError), (dict(q_weight=None), ValueError), (dict(k_weight=None), ValueError),
                     (dict(q_weight=w.bfloat16()), TypeError), (dict(q_weight=torch.ones(2, 64)), ValueError),
                     (dict(k_weight=torch.ones(4, 64)), ValueError), (dict(q_weight=torch.ones(128)[::2]), ValueError),
                     (dict(freqs=freqs.float()), TypeError), (dict(freqs=freqs[:31]), ValueError),
                     (dict(freqs=torch.ones(64, dtype=torch.float64)), ValueError), (dict(positions=None), ValueError),
                     (dict(positions=_i32(7)), ValueError), (dict(positions=_i32(8).long()), TypeError),
                     (dict(q=bf(8, 4, 128)[:, :, ::2]), ValueError), (dict(q_out=bf(8, 4, 32)), ValueError),
                     (dict(q_out=torch.zeros(8, 4, 64), k_out=bf(8, 2, 64)), TypeError), (dict(dtype=torch.float16), TypeError),
                     (dict(k=None), ValueError), (dict(), ValueError)):  # the last: host tensors
        with pytest.raises(err):
            fp4.qk_norm_rope(**{**good, **bad})


@pytest.mark.parametrize("eps", [1e-60, 1e-31, 0.0, -1e-6, 1e31, 1e300, float("nan"), float("inf")])
def test_binding_refuses_eps(fp4, eps):
    """1e-60 is 0 in fp32, which asks the library for no norm."""
    q, w = torch.zeros(8, 4, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="eps"):
        fp4.qk_norm_rope(q, None, None, None, w, None, eps)


def test_binding_refuses_pages(fp4):
    with pytest.raises(ValueError):
        fp4.KVPages(_i32(4), _i32(2), 24)
    with pytest.raises(ValueError):
        fp4.KVPages(_i32(4), _i32(3), 16)
    with pytest.raises(TypeError):
        fp4.KVPages(_i32(4).long(), _i32(2), 16)
    with pytest.raises(ValueError):
        fp4.KVPages(_i32(0), _i32(2), 16)
    with pytest.raises(ValueError, match="device"):
        fp4.KVPages(_i32(4), _i32(2), 16)
    pool = object.__new__(fp4.KVPages)  # a pool on the host, past its own check
    pool.free, pool.state, pool.pages, pool.page_size, pool.device = _i32(4), _i32(2), 4, 16, torch.device("cpu")
    good = dict(pages=pool, block_table=_i32(3, 5), seq_lens=_i32(3), new_lens=_i32(3), tokens=6)
    for bad, err in ((dict(block_table=_i32(3, 5).long()), TypeError), (dict(block_table=_i32(15)), ValueError),
                     (dict(seq_lens=_i32(4)), ValueError), (dict(new_lens=_i32(2)), ValueError),
                     (dict(new_lens=_i32(3).long()), TypeError), (dict(tokens=-1), ValueError), (dict(), ValueError),
                     (dict(out=fp4.KVPlan(_i32(6), _i32(6), None, None, _i32(3), _i32(2))), ValueError),
                     (dict(out=fp4.KVPlan(_i32(6).long(), _i32(5), None, None, _i32(3), _i32(2))), ValueError),
                     (dict(out=fp4.KVPlan(_i32(6).long(), _i32(6), _i32(3), None, _i32(3), _i32(2))), ValueError),
                     (dict(workspace=_i32(64)), ValueError)):
        with pytest.raises(err):
            fp4.kv_pages_extend(**{**good, **bad})
    with pytest.raises(ValueError):
        fp4.kv_pages_collect(pool, _i32(3, 5), _i32(4))
    good = dict(block_table=_i32(6, 5), seq_lens=_i32(6), parents=_i32(2, 3), page_size=16)
    for bad, err in ((dict(parents=_i32(2, 4)), ValueError), (dict(parents=_i32(6)), ValueError),
                     (dict(parents=_i32(2, 3).long()), TypeError), (dict(out=_i32(6, 6)), ValueError),
                     (dict(copies=_i32(6, 2)), ValueError), (dict(copies=_i32(5, 3)), ValueError),
                     (dict(copies=_i32(6, 3).long()), TypeError), (dict(), ValueError)):
        with pytest.raises(err):
            fp4.kv_pages_reorder(**{**good, **bad})


def test_binding_refuses_selection(fp4):
    good = dict(logits=torch.zeros(6, 100), scores=torch.zeros(2, 3))
    for bad, err in ((dict(logits=torch.zeros(5, 100)), ValueError), (dict(logits=torch.zeros(2, 3, 100)), ValueError),
                     (dict(logits=torch.zeros(6, 100).half()), TypeError), (dict(logits=torch.zeros(6, 200)[:, ::2]), ValueError),
                     (dict(scores=torch.zeros(6)), ValueError), (dict(scores=torch.zeros(2, 3).double()), TypeError),
                     (dict(scores=torch.zeros(3, 2).t()), ValueError), (dict(k=0), ValueError), (dict(k=65), ValueError),
                     (dict(done=torch.zeros(2, 3)), TypeError), (dict(done=torch.zeros(3, 2, dtype=torch.bool)), ValueError),
                     (dict(out=(torch.zeros(2, 3), _i32(2, 3), _i32(2, 4))), ValueError),
                     (dict(out=(torch.zeros(2, 3), _i32(2, 3))), ValueError),
                     (dict(out=(torch.zeros(2, 3), _i32(2, 3), torch.zeros(2, 3))), TypeError),
                     (dict(workspace=torch.zeros(4)), ValueError), (dict(), ValueError)):
        with pytest.raises(err):
            fp4.beam_select(**{**good, **bad})


def test_calls_go_to_the_tensors_device(fp4, monkeypatch):
    """The launch is made on the tensors' device and its current stream; prepare() records on the current one only."""
    now, seen = [0], []

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.old, now[0] = now[0], self.device

        def __exit__(self, *a):
            now[0] = self.old

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "device", On)

    def call(*args):
        seen.append((now[0], args))
        return 0

    fp4._run_on(0, call, 7)
    fp4._run_on(3, call, 8)
    assert seen == [(0, (7, 1000)), (3, (8, 1003))] and now == [0]
    with pytest.raises(ValueError, match="current device"):
        fp4.prepare(lambda: fp4._run_on(3, call, 9))
    assert fp4._recording is None
