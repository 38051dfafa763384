"""Beam selection on the GPU against the definition in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _fp4():
    import block_scaled_fp4_04_amd as fp4

    return fp4


def _totals(logits, scores, done, end):
    """float64 [batch, beams * vocab] on the host; what is not offered is -inf."""
    batch, beams = scores.shape
    z = logits.cpu().double().view(batch, beams, -1)
    d = z - z.amax(-1, keepdim=True)  # (differences first: logits near the type's lowest value would swallow the sum)
    t = scores.cpu().double()[..., None] + (d - torch.log(torch.exp(d).sum(-1, keepdim=True)))
    if done is not None:
        d = done.cpu().bool()
        t[d] = -math.inf
        t[..., end] = torch.where(d, scores.cpu().double(), t[..., end])
    return torch.where(t.isnan(), -math.inf, t).flatten(1)


def _check(logits, scores, k, done=None, end=0, exact=False, **kw):
    """A term e^-d of a row's sum is off by at most (1 + 2 d) 2^-23 of itself (v_exp_f32 and two roundings of its
    argument) and the terms that count have d < 30, so the sum's logarithm is within 2^-17, and a score its own rounding,
    2^-24 of it, more.  The choice is the definition's, but that totals nearer than that may stand in either
    order (`exact`: never)."""
    fp4 = _fp4()
    s, p, t = fp4.beam_select(logits, scores, k=k, done=done, end_token=end, **kw)
    batch, beams = scores.shape
    vocab = logits.shape[1]
    total = _totals(logits, scores, done, end)
    best, at = torch.sort(total, dim=-1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    real = best > -math.inf
    s, p, t = s.cpu(), p.cpu().long(), t.cpu().long()
    assert s.shape == p.shape == t.shape == (batch, k)
    assert torch.equal(s > -math.inf, real)
    assert bool((s[~real] == -math.inf).all()) and torch.equal((p * vocab + t)[~real], at[~real])  # in order
    tol = 2.0 ** -17 + 2.0 ** -24 * best.abs()
    assert bool(((s.double() - best).abs() <= tol)[real].all()), float((s.double() - best).abs()[real].max())
    flat = p * vocab + t
    same = flat == at
    assert bool((0 <= p).all()) and bool((p < beams).all()) and bool((t < vocab).all())
    if exact:
        assert bool(same[real].all()), (flat[~same & real], at[~same & real])
    chosen = total.gather(1, flat.clamp(min=0))
    assert bool(((chosen - best).abs() <= 2 * tol)[real].all())
    for b in range(batch):  # nothing twice
        assert flat[b].unique().numel() == k
    return s, p, t


def _logits(rows, vocab, dtype, seed, spread=2.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = spread * torch.randn(rows, vocab, device="cuda", generator=g)
    x[torch.rand(rows, vocab, device="cuda", generator=g) < 0.002] += 5.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,beams,vocab,k", [(1, 1, 1, 1), (1, 1, 7, 3), (2, 3, 5, 15), (3, 4, 257, 4), (1, 4, 32000, 4), (5, 2, 2047, 2), (4, 5, 2049, 10),
                                                 (2, 8, 8191, 16), (2, 7, 50003, 14), (1, 64, 1000, 64), (3, 16, 5000, 33), (40, 8, 131072, 8),
                                                 (65, 8, 40009, 16)])
def test_select(batch, beams, vocab, k, dtype):
    logits = _logits(batch * beams, vocab, dtype, vocab + k)
    scores = -10 * torch.rand(batch, beams, device="cuda", generator=torch.Generator("cuda").manual_seed(k))
    _check(logits, scores, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("off", range(8))
def test_rows_at_any_element(off, dtype):
    """Rows that begin anywhere and a stride that moves them: every alignment of a first and last vector."""
    rows, vocab = 6, 2050 + off
    room = torch.full((rows * (vocab + 13) + 40,), 1e4, dtype=dtype, device="cuda")  # read by mistake it would win
    logits = room[off:off + rows * (vocab + 13)].view(rows, vocab + 13)[:, :vocab]
    logits.copy_(_logits(rows, vocab, dtype, off))
    logits[:, 0], logits[:, -1] = 9.0, 9.5
    s, p, t = _check(logits, torch.zeros(2, 3, device="cuda"), 6)
    contiguous = logits.contiguous()
    assert all(torch.equal(a, b) for a, b in zip(_check(contiguous, torch.zeros(2, 3, device="cuda"), 6)[1:], (p, t)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [3, 500, 9000, 40000])
def test_ties(vocab, dtype):
    """Equal totals go to the lowest beam, then token: constant rows, equal beams, few levels."""
    fp4 = _fp4()
    zero = torch.zeros(1, 4, device="cuda")
    x = torch.zeros(4, vocab, dtype=dtype, device="cuda")
    s, p, t = fp4.beam_select(x, zero, k=6)
    want = [(i // vocab, i % vocab) for i in range(6)]
    assert p.tolist() == [[a for a, _ in want]] and t.tolist() == [[b for _, b in want]]
    row = torch.randint(0, 4, (vocab,), generator=torch.Generator().manual_seed(vocab)).to(dtype)
    x = row.cuda().expand(4, vocab).contiguous()
    order = torch.sort(row.double(), descending=True, stable=True).indices
    s, p, t = fp4.beam_select(x, zero, k=8)
    top = int((row == row.max()).sum())
    want = [(b, int(order[i])) for b in range(4) for i in range(min(top, 8))][:8]  # of equal rows, beam 0's first
    assert list(zip(p[0].tolist(), t[0].tolist()))[:len(want)] == want
    s, p, t = fp4.beam_select(x[:1], zero[:, :1], k=min(64, vocab))
    assert t[0].tolist() == order[:min(64, vocab)].tolist()
    # -0 and 0 are equal
    x = torch.zeros(1, vocab, dtype=dtype, device="cuda")
    x[0, 0] = -0.0
    assert fp4.beam_select(x, zero[:, :1], k=2)[2].tolist() == [[0, 1]]


@pytest.mark.parametrize("vocab", [40, 3000, 20000])
def test_masked_and_nonfinite(vocab):
    fp4 = _fp4()
    inf = math.inf
    x = _logits(8, vocab, torch.float32, 3)
    scores = torch.tensor([[0.0, -1.0, -inf, -2.0], [-1.0, -1.0, -1.0, -1.0]], device="cuda")
    x[0, 5:] = -inf                                   # five tokens are left
    x[1, :] = -inf                                    # nothing
    x[3, 7] = float("nan")                            # spoils its row
    x[4, 11] = inf
    x[5, :] = torch.finfo(torch.float32).min          # all equal, at the lowest value
    x[6, ::2] = torch.finfo(torch.float32).min
    _check(x, scores, 8)
    _check(x, scores, 3)
    s, p, t = _check(x, torch.full((2, 4), -inf, device="cuda"), 5)
    assert bool((s == -inf).all())
    # one token alone, at the far end
    y = torch.full((4, vocab), -inf, dtype=torch.bfloat16, device="cuda")
    y[2, vocab - 1] = -3.0
    s, p, t = fp4.beam_select(y, torch.zeros(1, 4, device="cuda"))
    assert t.tolist() == [[vocab - 1, 0, 1, 2]] and p.tolist() == [[2, 0, 0, 0]] and s[0, 0] == 0.0


@pytest.mark.parametrize("kind", [torch.bool, torch.uint8])
def test_ended_beams(kind):
    fp4 = _fp4()
    batch, beams, vocab = 6, 5, 9001
    x = _logits(batch * beams, vocab, torch.bfloat16, 9)
    g = torch.Generator("cuda").manual_seed(2)
    scores = -6 * torch.rand(batch, beams, device="cuda", generator=g)
    done = (torch.rand(batch, beams, device="cuda", generator=g) < 0.4)
    done[0] = True
    done[1] = False
    x[done.flatten()] = float("nan")  # not read
    d = done.to(kind) * (3 if kind == torch.uint8 else 1) if kind == torch.uint8 else done
    for k in (5, 10):
        _check(x, scores, k, done=d, end=vocab - 1)
    s, p, t = fp4.beam_select(x, scores, k=10, done=d, end_token=77)
    assert t[0].tolist() == [77] * 5 + [0, 1, 2, 3, 4] and p[0, 5:].tolist() == [0] * 5
    order = torch.sort(scores[0], descending=True, stable=True)
    assert p[0, :5].tolist() == order.indices.tolist() and torch.equal(s[0, :5], order.values)


def test_small_differences_of_low_scores():
    """Logits of neighbouring fp32 values under scores where fp32 sums would merge them."""
    fp4 = _fp4()
    base = torch.full((1, 4000), -20.0, device="cuda")
    eps = 2.0 ** -23
    at = [3000, 17, 2999, 5]
    for i, a in enumerate(at):
        base[0, a] = 1.0 + (4 - i) * eps
    s, p, t = fp4.beam_select(base, torch.full((1, 1), -400.0, device="cuda"), k=4)
    assert t.tolist() == [at]


def test_large_logits():
    """Differences past the range of the exponential, and rows whose best are far apart between parts."""
    x = _logits(3, 30000, torch.float32, 4) * 50
    x[0, 29999] = 1e30
    x[1, 12345] = -1e30
    x[2] = x[2] * 1e30
    _check(x, torch.tensor([[-1.0, -2.0, -3.0]], device="cuda"), 6)


def test_captured_with_one_workspace():
    fp4 = _fp4()
    batch, beams, vocab, k = 3, 4, 5001, 8
    ws = fp4.beam_select_workspace(batch, beams, vocab, k)
    x, scores = _logits(12, vocab, torch.bfloat16, 1), torch.zeros(batch, beams, device="cuda")
    out = tuple(torch.empty(batch, k, dtype=d, device="cuda") for d in (torch.float32, torch.int32, torch.int32))
    fp4.beam_select(x, scores, k=k, workspace=ws)
    graphs = []
    for _ in range(2):  # two graphs share the workspace, replayed one behind the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = fp4.beam_select(x, scores, k=k, workspace=ws, out=out)
        assert got is out
        graphs.append(g)
    for i in range(4):
        x.copy_(_logits(12, vocab, torch.bfloat16, 30 + i))
        scores.copy_(-torch.rand(batch, beams))
        graphs[i % 2].replay()
        want = fp4.beam_select(x, scores, k=k)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_many_parts():
    """A vocabulary of many parts, few rows; the best at a part's first and last place."""
    vocab = 1 << 20
    x = torch.zeros(2, vocab, dtype=torch.bfloat16, device="cuda")
    at = [0, 2047, 2048, 8191, 8192, 524287, vocab - 1]
    for i, a in enumerate(at):
        x[0, a], x[1, a] = 20.0 - i, 13.0 + i / 2
    _check(x, torch.tensor([[0.0, -0.25]], device="cuda"), 12)


def test_rows_past_4gib():
    rows, vocab, ld = 4, 5000, 3 * (1 << 28) + 1
    room = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = room.as_strided((rows, vocab), (ld, 1))
    x.copy_(_logits(rows, vocab, torch.bfloat16, 3))
    scores = -torch.rand(2, 2, device="cuda")
    got, want = _check(x, scores, 6), _check(x.contiguous(), scores, 6)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_recorded_and_on_another_stream():
    fp4 = _fp4()
    x, scores = _logits(6, 3001, torch.bfloat16, 1), torch.zeros(2, 3, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = []
        call = fp4.prepare(lambda: got.extend(fp4.beam_select(x, scores)))
        x.copy_(_logits(6, 3001, torch.bfloat16, 2))
        call()
        want = fp4.beam_select(x, scores)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_steps_of_every_size():
    """Lengths around the borders of a vector, a group and a part, the best tokens at their ends."""
    fp4 = _fp4()
    for dtype, per in ((torch.bfloat16, 8), (torch.float32, 4)):
        for edge in (per, 64 * per, 256 * per, 1024 * per, 4096 * per):
            for vocab in (edge - 1, edge, edge + 1):
                x = _logits(2, vocab, dtype, vocab)
                x[0, -1], x[1, 0], x[1, vocab // 2] = 12.0, 12.5, 13.0
                _check(x, torch.tensor([[0.0, -0.3]], device="cuda"), 5)


def test_sorted_rows():
    """Logits in rising and falling order: all of the best in one lane's, one wave's, one part's reach."""
    for dtype in (torch.bfloat16, torch.float32):
        for vocab in (700, 20000, 70000):
            up = torch.linspace(-9, 9, vocab, device="cuda")
            _check(torch.stack([up, up.flip(0), up.abs()]).to(dtype), torch.tensor([[0.0, -0.5, -0.1]], device="cuda"), 48)


def test_fewer_continuations_than_places():
    """Masked rows, dead and ended beams: what is left comes in the order of beam and token, around what was chosen."""
    inf = math.inf
    for vocab in (6, 70, 5000):
        x = torch.full((8, vocab), -inf, device="cuda")
        x[0, 0], x[0, 2], x[1, 1], x[2, 5], x[3, vocab - 1] = 1.0, 2.0, 0.5, 0.0, 3.0
        x[5] = 1.0
        scores = torch.tensor([[0.0, -1.0, -inf, -0.5], [-inf, -inf, float("nan"), -2.0]], device="cuda")
        done = torch.tensor([[False, False, False, False], [False, False, False, True]], device="cuda")
        for k in (1, 4, 5, 16, 24):
            _check(x, scores, k, done=done, end=2)
            _check(x.bfloat16(), scores, k, done=done, end=2)


@pytest.mark.parametrize("beams,vocab", [(1, 50), (8, 40000), (40, 300)])
def test_scores_in_place(beams, vocab):
    fp4 = _fp4()
    x = _logits(5 * beams, vocab, torch.bfloat16, vocab)
    scores = -9 * torch.rand(5, beams, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    want = fp4.beam_select(x, scores)
    out = (scores, torch.empty_like(want[1]), torch.empty_like(want[2]))
    fp4.beam_select(x, scores, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_logits_past_the_caches():
    """Over 96 MB, rows at odd elements: the same bits as from aligned rows, and the definition's choice."""
    batch, beams, vocab = 130, 4, 100003
    x = _logits(batch * beams, vocab, torch.bfloat16, 6)
    scores = -9 * torch.rand(batch, beams, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    room = torch.zeros(batch * beams, vocab + 5, dtype=torch.bfloat16, device="cuda")
    room[:, :vocab] = x
    got = _check(x, scores, 8)
    assert all(torch.equal(a, b) for a, b in zip(got, _check(room[:, :vocab], scores, 8)))
    part = [t.cpu() for t in _fp4().beam_select(x[:4 * beams], scores[:4], k=8)]  # below that size
    assert all(torch.equal(a, b[:4]) for a, b in zip(part[1:], got[1:]))


@pytest.mark.parametrize("batch,beams,vocab,k,dtype", [(270, 4, 50001, 8, torch.bfloat16), (310, 7, 12503, 14, torch.float32)])
def test_many_short_rows_past_the_caches(batch, beams, vocab, k, dtype):
    """Over 96 MB in rows that few waves read, some of them ended: the definition's choice, alone and among others."""
    x = _logits(batch * beams, vocab, dtype, 7)
    g = torch.Generator("cuda").manual_seed(5)
    scores = -9 * torch.rand(batch, beams, device="cuda", generator=g)
    done = torch.rand(batch, beams, device="cuda", generator=g) < 0.2
    got = _check(x, scores, k, done=done, end=3)
    one = [t.cpu() for t in _fp4().beam_select(x[:beams], scores[:1], k=k, done=done[:1], end_token=3)]
    assert all(torch.equal(a, b[:1]) for a, b in zip(one[1:], got[1:]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wide", [False, True])
def test_best_far_above_where_a_row_begins(dtype, wide):
    """Peaks (one value, or a plateau of 4096) from 0 to 90 above a row's first values, anywhere in it, in rows of which a wave
    walks several groups: a row's sum is within the documented 2^-18 wherever its largest terms stand, and a score's own
    rounding is 2^-24 of it more.  The peaks' tokens are the definition's."""
    rows, vocab, k = 1024, 16384, 4
    g = torch.Generator("cuda").manual_seed(11)
    x = 16 * torch.rand(rows, vocab, device="cuda", generator=g) - 8
    up = torch.linspace(0, 90, rows, device="cuda")
    if wide:
        x[:, vocab // 2:vocab // 2 + 4096] += up[:, None]
    else:
        at = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
        x[torch.arange(rows, device="cuda"), at] = 8 + up
    x = x.to(dtype)
    scores = torch.zeros(rows, 1, device="cuda")
    s, p, t = _fp4().beam_select(x, scores, k=k)
    best, order = torch.sort(_totals(x, scores, None, 0), dim=-1, descending=True, stable=True)
    err = (s.cpu().double() - best[:, :k]).abs() - 2.0 ** -24 * best[:, :k].abs()
    assert float(err.max()) <= 2.0 ** -18, (float(err.max()) * 2 ** 18, int((err > 2.0 ** -18).any(1).sum()))
    assert torch.equal(t.cpu().long(), order[:, :k])  # (one beam: the order is that of its logits)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", [-1e30, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("vocab", [3, 7, 300, 20000, 140000])
def test_scores_that_swallow_logits(vocab, low, dtype):
    """Beams held back by a score beside which 64 bits hold no difference of logits: their totals are all equal, so they come by
    beam, and within a beam in the order of its logits, then of its tokens."""
    fp4 = _fp4()
    x = _logits(4, vocab, dtype, vocab).cpu()
    x[1] = x[1].flip(0)
    x[2, : vocab // 2] = x[2, 0]  # equal logits: the lower token
    order = [torch.sort(r.double(), descending=True, stable=True).indices.tolist() for r in x]
    for k in (4, min(64, 4 * vocab)):
        s, p, t = fp4.beam_select(x.cuda(), torch.full((1, 4), low, device="cuda"), k=k)
        want = [(b, v) for b in range(4) for v in order[b][:64]][:k]
        assert list(zip(p[0].tolist(), t[0].tolist())) == want, k
        assert bool((s == torch.tensor(low)).all())
    if vocab < 16:  # fewer continuations of the one live beam, and of an ended one, than places
        scores = torch.tensor([[low, -1.0, low, low]], device="cuda")
        done = torch.tensor([[False, False, False, True]], device="cuda")
        p, t = fp4.beam_select(x.cuda(), scores, k=3 * vocab + 1, done=done, end_token=2)[1:]
        want = [(b, v) for b in (1, 0, 2) for v in order[b]] + [(3, 2)]
        assert list(zip(p[0].tolist(), t[0].tolist())) == want


def test_logits_nearer_than_a_total_tells():
    """One beam's logits that differ by less than the last bit of their totals, in one part of the row and in two."""
    fp4 = _fp4()
    for at in ([30, 17, 29, 5], [39000, 17, 20001, 5]):
        x = torch.full((1, 40000), -20.0, device="cuda")
        for i, a in enumerate(at):
            x[0, a] = 0.25 - i * 2.0 ** -26
        s, p, t = fp4.beam_select(x, torch.full((1, 1), -1e9, device="cuda"), k=4)
        assert t.tolist() == [at]
        y = torch.full((1, 40000), -50.0, device="cuda")
        y[0, 100] = 9.0
        for i, a in enumerate(at):
            y[0, a] = 1e-20 * (4 - i)
        assert fp4.beam_select(y, torch.zeros(1, 1, device="cuda"), k=5)[2].tolist() == [[100] + at]
