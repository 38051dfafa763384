"""The generate loop as a whole: pages, layers, selection and reordering together, eager and captured."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("beam_search", os.path.join(ROOT, "examples", "beam_search.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt,beams,prompts,steps,page", [("bf16", 4, (37, 5, 64), 20, 16), ("bf16", 3, (1, 16), 36, 16), ("mxfp8", 8, (33, 47), 12, 32),
                                                          ("bf16", 1, (9,), 6, 16), ("mxfp4", 2, (20, 31, 32, 1), 9, 16)])
def test_beams_hold_their_own_texts(example, fmt, beams, prompts, steps, page):
    """The first layer's keys depend on a beam's tokens and positions alone: whatever was shared, moved, copied and
    given back, the rows that a beam's table names are those of its text.  bf16: the projection's rows may be
    rounded from sums in another order (2^-7 of the row's largest value, after the norm); coarser formats: one
    step of the element (an eighth, a half) of the block's largest value more."""
    import block_scaled_fp4_04_amd as fp4

    texts, scores, search = example.run(fmt, prompts, beams, steps, page=page)
    model = search.model
    assert bool(torch.isfinite(scores).all()) and bool((scores[:, :-1] >= scores[:, 1:]).all())
    step = {"bf16": 0.0, "mxfp8": 2.0 ** -3, "mxfp4": 2.0 ** -1}[fmt]
    lens = search.lens.tolist()
    for b, group in enumerate(texts):
        for j, text in enumerate(group):
            row = b * beams + j
            n = lens[row]
            assert n == len(text) - 1 == prompts[b] + steps - 1
            cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            k, v = fp4.kv_cache_read(search.caches[0], search.table[row:row + 1], cu, n, dtype=torch.float32)
            x = model.embedding[torch.tensor(text[:n], device="cuda")]
            _, kk, vv = model.projected(0, x)
            at = torch.arange(n, dtype=torch.int32, device="cuda")
            want = fp4.qk_norm_rope(kk, None, at, model.freqs, model.layers[0][5], eps=1e-6, dtype=torch.float32)[0]
            for got, ref in ((k, want), (v, vv.float())):
                lim = (2.0 ** -7 + step) * ref.abs().amax(-1, keepdim=True)
                assert bool(((got - ref).abs() <= lim).all()), (row, float(((got - ref).abs() / lim).max()))
    # every page is held by a beam or free, and a partly filled one by one beam
    held, last = set(), []
    for row, n in zip(search.table.tolist(), lens):
        used = row[:-(-n // page)]
        held |= set(used)
        if n % page:
            last.append(used[-1])
    free, refused = search.pool.state.tolist()
    assert refused == 0 and len(last) == len(set(last))
    assert sorted(held | set(search.pool.free[:free].tolist())) == list(range(search.pool.pages))
    assert len(held) + free == search.pool.pages


def test_captured_is_eager(example):
    one = example.run("mxfp8", (20, 7), 3, 15, graph=True)
    two = example.run("mxfp8", (20, 7), 3, 15, graph=False)
    assert one[0] == two[0] and torch.equal(one[1], two[1])


def test_beams_end(example, monkeypatch):
    """Beams that end keep their score and are carried along."""
    texts, scores, search = example.run("bf16", (12, 3), 4, 10, graph=False)
    end = texts[0][0][-1]
    monkeypatch.setattr(example, "END", end)
    texts, scores, search = example.run("bf16", (12, 3), 4, 14, graph=False)
    for group, row in zip(texts, search.done.tolist()):
        for text, done in zip(group, row):
            made = text[-14:]
            if end in made:
                assert done and set(made[made.index(end):]) == {end}
            else:
                assert not done
