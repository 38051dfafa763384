"""Pages dealt, taken back and reordered on the device, against a plain allocator on the host."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _fp4():
    import block_scaled_fp4_04_amd as fp4

    return fp4


class Host:
    """The definition, one sequence and one token at a time."""

    def __init__(self, free, count, table, page):
        self.free, self.count, self.table, self.page, self.refused = list(free), count, [list(r) for r in table], page, 0

    def extend(self, lens, new, tokens):
        lens, slots, positions, cu_q, cu_k = list(lens), [], [], [0], [0]
        short = False
        want = 0  # pages asked for so far
        taken, begin = 0, 0
        for b, (held, n) in enumerate(zip(list(lens), new)):
            n = max(n, 0)
            begin += n
            width = len(self.table[b])
            fits = held >= 0 and held + n <= width * self.page and begin <= tokens
            have = -(-held // self.page) if fits else 0
            need = -(-(held + n) // self.page) - have if fits else 0
            want += need
            given = fits and (need == 0 or want <= self.count)
            if given:
                for i in range(need):
                    self.table[b][have + i] = self.free[self.count - 1 - (want - need) - i]
                taken = want if need else taken
                lens[b] = held + n
            elif n:
                self.refused += 1
            for i in range(n):
                pos = held + i
                positions.append(pos)
                slots.append(self.table[b][pos // self.page] * self.page + pos % self.page if given else -1)
            cu_q.append(min(begin, tokens))
            cu_k.append(cu_k[-1] + max(lens[b], 0))
        self.count -= taken
        slots += [-1] * (tokens - len(slots))
        positions += [0] * (tokens - len(positions))
        return lens, slots[:tokens], positions[:tokens], cu_q, cu_k

    def collect(self, lens):
        held = {p for r, n in zip(self.table, lens) for p in r[:min(len(r), -(-max(n, 0) // self.page))]}
        ids = [p for p in range(len(self.free)) if p not in held]
        self.free[:len(ids)] = ids
        self.count = len(ids)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _start(fp4, seqs, width, page, pages, lens, seed, wide=0):
    """A pool and a table that hold `lens`, on both sides."""
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = [[-1] * width for _ in range(seqs)]
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[b][i] = order.pop()
    count = len(order)
    free = order + [-7] * (pages - count)
    host = Host(free, count, table, page)
    room = torch.full((seqs, width + wide), -9, dtype=torch.int32, device="cuda")
    dev = room[:, :width]
    dev.copy_(_i32(table).view(seqs, width))
    return host, fp4.KVPages(_i32(free), _i32([count, 0]), page), dev, room


def _equal(host, pool, table, what):
    assert pool.state.tolist() == [host.count, host.refused], what
    assert pool.free.tolist() == host.free, what
    assert table.tolist() == host.table, what


@pytest.mark.parametrize("seqs,width,page,most_held,most_new,share", [
    (1, 1, 16, 0, 1, 1.0), (1, 9, 16, 40, 100, 1.0), (64, 20, 64, 900, 1, 1.0), (64, 20, 16, 300, 1, 0.3), (65, 8, 32, 120, 40, 0.6),
    (1000, 4, 16, 40, 3, 0.5), (1025, 5, 16, 40, 2, 0.8), (2500, 6, 16, 60, 5, 0.9), (7, 300, 16, 1000, 3500, 0.7), (3, 40, 256, 9000, 5000, 1.0)])
@pytest.mark.parametrize("in_place", [True, False])
def test_extend(seqs, width, page, most_held, most_new, share, in_place):
    fp4 = _fp4()
    rng = torch.Generator().manual_seed(seqs + page)
    cap = width * page
    lens = [min(cap, int(x * (most_held + 1))) for x in torch.rand(seqs, generator=rng).tolist()]
    new = [1 if most_new == 1 else int(x * (most_new + 1)) for x in torch.rand(seqs, generator=rng).tolist()]
    for b in range(0, seqs, 11):
        lens[b], new[(b + 3) % seqs] = lens[b] // page * page, 0  # whole pages, nothing new
    if seqs > 20:
        new[13] = -4           # counts as 0
        lens[17] = cap - 1     # too wide with more than one
        new[17] = 5
    need = sum(-(-(a + max(n, 0)) // page) - -(-a // page) for a, n in zip(lens, new))
    held = sum(-(-a // page) for a in lens)
    for extra in (0, 7):  # slots past the last token
        host, pool, table, room = _start(fp4, seqs, width, page, held + int(need * share) + 1, lens, 5, wide=3)
        tokens = sum(max(n, 0) for n in new) + extra
        dl = _i32(lens)
        free, state = pool.free.clone(), pool.state.clone()
        plan = fp4.kv_pages_extend(pool, table, dl, _i32(new), tokens, in_place=in_place)
        want = host.extend(lens, new, tokens)
        assert (plan.seq_lens is dl) == in_place and (plan.state is pool.state) == in_place
        if not in_place:
            assert torch.equal(pool.state, state) and dl.tolist() == lens
            pool.state.copy_(plan.state)
        for got, ref, name in zip((plan.seq_lens, plan.slots, plan.positions, plan.cu_q, plan.cu_k), want,
                                  ("lens", "slots", "positions", "cu_q", "cu_k")):
            assert got.tolist() == ref, name
        assert plan.slots.dtype == torch.int64 and torch.equal(pool.free, free)
        _equal(host, pool, table, "extend")
        assert bool((room[:, width:] == -9).all())


def test_extend_refuses_lengths():
    """Lengths and counts that no sequence can have, tokens past the arrays: refused, the others served."""
    fp4 = _fp4()
    lens, new = [-3, 5, 2 ** 31 - 1, 0, 20, 3, 0], [2, 3, 2 ** 31 - 1, 4, 2 ** 31 - 1, 0, 5]
    host, pool, table, _ = _start(fp4, 7, 4, 16, 12, [0, 5, 0, 0, 20, 3, 0], 3)
    dl = _i32(lens)
    plan = fp4.kv_pages_extend(pool, table, dl, _i32(new), 9)
    assert dl.tolist() == [-3, 8, 2 ** 31 - 1, 0, 20, 3, 0]  # b = 2 on lies past the 9 tokens
    assert pool.state.tolist() == [12 - 1 - 2 - 1, 5]
    slots = plan.slots.tolist()
    page = table[1, 0].item()
    assert slots == [-1, -1] + [page * 16 + i for i in (5, 6, 7)] + [-1] * 4
    assert plan.cu_q.tolist() == [0, 2, 5, 9, 9, 9, 9, 9]
    assert plan.cu_k.tolist()[:3] == [0, 0, 8] and plan.cu_k.tolist()[3:] == [2 ** 31 - 1] * 5
    # a pool whose count is nonsense deals nothing outside itself
    for count in (-5, 1 << 30):
        pool.state.copy_(_i32([count, 0]))
        pool.free.fill_(3)
        dl = _i32([0, 0, 0, 0, 0, 0, 0])
        fp4.kv_pages_extend(pool, table, dl, _i32([1] * 7), 7)
        assert dl.tolist() == ([0] * 7 if count < 0 else [1] * 7)
    # a page id that is nonsense gives no slot
    table.fill_(99)
    plan = fp4.kv_pages_extend(pool, table, _i32([3] * 7), _i32([1] * 7), 7)
    assert plan.slots.tolist() == [-1] * 7


def test_extend_nothing():
    fp4 = _fp4()
    _, pool, table, _ = _start(fp4, 3, 2, 16, 5, [0, 4, 16], 1)
    dl = _i32([0, 4, 16])
    plan = fp4.kv_pages_extend(pool, table, dl, _i32([0, 0, 0]), 0)
    assert plan.slots.numel() == 0 and dl.tolist() == [0, 4, 16] and plan.cu_k.tolist() == [0, 0, 4, 20]
    plan = fp4.kv_pages_extend(pool, table, dl, _i32([0, 0, 0]), 5, offsets=False)
    assert plan.cu_q is None and plan.slots.tolist() == [-1] * 5 and plan.positions.tolist() == [0] * 5


@pytest.mark.parametrize("seqs,width,page,pages,longest", [(1, 1, 16, 1, 16), (1, 40, 16, 31, 0), (5, 7, 32, 40, 200), (64, 64, 16, 5000, 1000),
                                                           (300, 200, 16, 70000, 3200), (40, 900, 256, 40000, 200000),
                                                           (16, 3000, 16, 600000, 40000), (9000, 1, 16, 9100, 16),
                                                           (700, 23, 16, 20000, 360), (5, 65, 16, 400, 1040), (3, 400, 16, 1300, 6400)])
def test_collect(seqs, width, page, pages, longest):
    fp4 = _fp4()
    rng = torch.Generator().manual_seed(pages)
    lens = [min(width * page, int(x * (longest + 1))) for x in torch.rand(seqs, generator=rng).tolist()]
    host, pool, table, _ = _start(fp4, seqs, width, page, pages, lens, 2, wide=1)
    now = [0 if i % 3 == 1 else n // 2 if i % 3 == 2 else n for i, n in enumerate(lens)]
    if seqs > 4 and width >= 4:  # shared pages, entries outside the pool, a length past the row
        host.table[3][:4] = host.table[0][:4]
        host.table[4][:2] = [-1, pages]
        now[4] = max(now[4], 2 * page)
        now[0] = 4 * page
        table.copy_(_i32(host.table))
    lens_dev = _i32(now)
    if seqs > 4:
        lens_dev[3] = 2 ** 31 - 1
        now[3] = width * page
    fp4.kv_pages_collect(pool, table, lens_dev)
    host.collect(now)
    host.free = [p if p is not None else None for p in host.free]
    assert pool.state.tolist() == [host.count, 0]
    assert pool.free[:host.count].tolist() == host.free[:host.count]
    assert pool.free.tolist() == host.free


def test_generate_and_release():
    """Steps of a serving loop: sequences grow, end and begin again; every page is held once or free."""
    fp4 = _fp4()
    seqs, width, page, pages = 9, 12, 16, 60
    host, pool, table, _ = _start(fp4, seqs, width, page, pages, [0] * seqs, 4)
    lens, dl = [0] * seqs, _i32([0] * seqs)
    rng = torch.Generator().manual_seed(6)
    for step in range(40):
        new = (torch.randint(0, 30, (seqs,), generator=rng) if step % 5 == 0 else torch.ones(seqs, dtype=torch.long)).tolist()
        fp4.kv_pages_extend(pool, table, dl, _i32(new), sum(new))
        lens = host.extend(lens, new, sum(new))[0]
        assert dl.tolist() == lens
        _equal(host, pool, table, step)
        if step % 7 == 6:
            for b in (step % seqs, (step * 5) % seqs):
                lens[b] = 0
                dl[b] = 0
            fp4.kv_pages_collect(pool, table, dl)
            host.collect(lens)
            _equal(host, pool, table, step)
            held = [p for r, n in zip(host.table, lens) for p in r[:-(-n // page)]]
            assert sorted(held + host.free[:host.count]) == list(range(pages))


def test_extend_captured():
    fp4 = _fp4()
    seqs, width, page = 20, 6, 16
    lens = list(range(0, 60, 3))
    host, pool, table, _ = _start(fp4, seqs, width, page, 100, lens, 8)
    dl, one = _i32(lens), _i32([1] * seqs)
    plan = fp4.kv_pages_extend(pool, table, dl, one, seqs)
    lens = host.extend(lens, [1] * seqs, seqs)[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4.kv_pages_extend(pool, table, dl, one, seqs, out=plan)
        fp4.kv_pages_collect(pool, table, dl)
    for i in range(5):
        graph.replay()
        lens, slots, positions, cu_q, cu_k = host.extend(lens, [1] * seqs, seqs)
        host.collect(lens)
        assert (plan.slots.tolist(), plan.positions.tolist(), dl.tolist()) == (slots, positions, lens), i
        _equal(host, pool, table, i)
        torch.zeros(1000, device="cuda").sum().item()


def _reorder_host(table, lens, parents, page):
    """(new rows, copies) of one group."""
    beams = len(table)
    parents = [p if 0 <= p < beams else j for j, p in enumerate(parents)]
    n = lens[0]
    at, off = n // page, n % page
    spare = [i for i in range(beams) if i not in parents]
    rows, copies, m = [], [], 0
    for j, p in enumerate(parents):
        row = list(table[j])
        row[:-(-n // page)] = table[p][:-(-n // page)]
        rec = [-1, -1, 0]
        if p in parents[:j]:
            if off:
                rec = [table[p][at], table[spare[m]][at], off]
                row[at] = table[spare[m]][at]
            m += 1
        rows.append(row)
        copies.append(rec)
    return rows, copies


@pytest.mark.parametrize("batch,beams,width,page,n", [(1, 1, 1, 16, 5), (1, 2, 3, 16, 16), (2, 4, 5, 16, 33), (3, 8, 40, 32, 1279), (2, 64, 9, 64, 511),
                                                      (2, 5, 700, 16, 11199), (2, 5, 700, 16, 4097), (1, 3, 256, 16, 4096), (5, 6, 300, 16, 0),
                                                      (300, 4, 3, 256, 700)])
def test_reorder(batch, beams, width, page, n):
    fp4 = _fp4()
    rows = batch * beams
    rng = torch.Generator().manual_seed(n + beams)
    table = torch.randperm(rows * width, generator=rng).to(torch.int32).view(rows, width)
    for how in range(4):
        parents = torch.randint(0, beams, (batch, beams), generator=rng, dtype=torch.int32)
        if how == 1:
            parents[:] = beams - 1              # all from the last
        elif how == 2:
            parents[:] = torch.arange(beams)    # nothing changes
        elif how == 3 and beams > 2:
            parents[0, 0], parents[-1, 2] = -1, beams  # keep their own
        want, copies = [], []
        for b in range(batch):
            r, c = _reorder_host(table[b * beams:(b + 1) * beams].tolist(), [n] * beams, parents[b].tolist(), page)
            want += r
            copies += c
        lens = _i32([n] * rows)
        room = torch.full((rows, width + 5), -9, dtype=torch.int32, device="cuda")
        dev = room[:, :width]
        dev.copy_(table)
        out = dev.clone().fill_(-3)
        assert fp4.kv_pages_reorder(dev, lens, parents.cuda(), page, out=out).tolist() == copies
        live = -(-n // page)
        assert out[:, :live].tolist() == [r[:live] for r in want] and bool((out[:, live:] == -3).all())
        assert torch.equal(dev.cpu(), table)
        got = torch.full((rows, 3), 5, dtype=torch.int32, device="cuda")
        assert fp4.kv_pages_reorder(dev, lens, parents.cuda(), page, copies=got) is got
        assert got.tolist() == copies and dev.tolist() == want
        assert bool((room[:, width:] == -9).all())


def test_reorder_bad_lengths_stay_inside():
    """Lengths that no group can have: results are unspecified, the memory around the rows stays."""
    fp4 = _fp4()
    room = torch.arange(8 * 12, dtype=torch.int32, device="cuda").view(8, 12)
    before = room.clone()
    table = room[1:7, 2:6]
    lens = _i32([5, 2 ** 31 - 1, -4, 64, 65, 33])
    copies = fp4.kv_pages_reorder(table, lens, _i32([[1, 1, 0], [2, 1, 1]]), 16)
    assert copies.shape == (6, 3)
    mask = torch.ones_like(room, dtype=torch.bool)
    mask[1:7, 2:6] = False
    assert torch.equal(room[mask], before[mask])


@pytest.mark.parametrize("beams,width,page", [(4, 5, 16), (8, 300, 16), (64, 3, 32)])
@pytest.mark.parametrize("aside", [False, True])
def test_reorder_uneven_lengths_touch_no_other_page(beams, width, page, aside):
    """A pool that ran out under some beams leaves lengths that differ and, past them, entries of earlier sequences:
    none is copied into or from, or comes within a row's own or its parent's length."""
    fp4 = _fp4()
    batch, rows = 5, 5 * beams
    rng = torch.Generator().manual_seed(beams)
    for _ in range(6):
        lens = torch.randint(0, width * page + 1, (rows,), generator=rng, dtype=torch.int32)
        short = torch.randint(0, 2, (rows,), generator=rng, dtype=torch.int32)
        lens[beams:] = lens[beams:].view(batch - 1, beams)[:, :1].repeat(1, beams).flatten()  # off by a token at most
        lens[beams:] = (lens[beams:] - short[beams:]).clamp(min=0)
        held = torch.arange(width) < -(-lens // page)[:, None]
        own = torch.arange(rows * width, dtype=torch.int32).view(rows, width)
        table = torch.where(held, own, 100000 + own)                       # from 100000 on: others' pages
        parents = torch.randint(0, beams, (batch, beams), generator=rng, dtype=torch.int32)
        dev = table.cuda()
        out = torch.full_like(dev, 200000) if aside else dev
        copies = fp4.kv_pages_reorder(dev, lens.cuda(), parents.cuda(), page, out=out).cpu()
        assert int(copies[:, :2].max()) < 100000
        of = (torch.arange(batch)[:, None] * beams + parents).flatten().long()
        live = held | held[of]
        assert int(out.cpu()[live].max()) < 100000
        full = torch.arange(width) < (lens[of] // page)[:, None]           # the parent's full pages, whatever the lengths
        assert torch.equal(out.cpu()[full], table[of][full])
        to = copies[copies[:, 1] >= 0, 1]
        assert to.unique().numel() == to.numel()
        assert torch.equal(lens[to.long() // width] // page, to % width) and bool((lens[to.long() // width] % page > 0).all())


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("dim,heads,page", [(64, 1, 16), (128, 3, 64), (256, 2, 256)])
def test_copy(fmt, dim, heads, page):
    fp4 = _fp4()
    pages = 14
    ts = [torch.rand(heads, device="cuda") for _ in range(2)] if fmt == "nvfp4" else [None, None]
    cache = fp4.KVCache.alloc(fmt, pages, heads, page, dim, "cuda", *ts)
    parts = [t for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales) if t is not None]
    g = torch.Generator("cuda").manual_seed(3)
    for t in parts:
        b = t.view(torch.uint8)
        b.copy_(torch.randint(0, 256, b.shape, device="cuda", generator=g, dtype=torch.uint8))
    before = [t.clone() for t in parts]
    copies = [[0, 1, page], [0, 2, page - 1], [3, 4, 1], [5, 6, page // 2 + 3], [-1, -1, 0], [7, -1, 4], [-1, 7, 4], [7, pages, 4], [pages, 8, 4],
              [9, 10, 0], [9, 11, -3], [12, 12, 5], [12, 13, page + 9]]
    fp4.kv_cache_copy(cache, _i32(copies))
    want = [t.clone() for t in before]
    for src, dst, n in copies:
        if src < 0 or dst < 0 or src >= pages or dst >= pages or n <= 0:
            continue
        for t, old in zip(want, before):
            n = min(n, page)
            if t.shape[2] == page and t.shape[3] != page or t is want[0] or t is want[1]:
                t[dst, :, :n] = old[src, :, :n]
            else:
                t[dst, :, :, :n] = old[src, :, :, :n]
    for got, ref in zip(parts, want):
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
    fp4.kv_cache_copy(cache, torch.empty((0, 3), dtype=torch.int32, device="cuda"))


def test_recorded_calls():
    """prepare() replays a step's planning: pages dealt, rows reordered, pages taken back."""
    fp4 = _fp4()
    host, pool, table, _ = _start(fp4, 4, 6, 16, 40, [15, 15, 31, 31], 3)
    lens, one = _i32([15, 15, 31, 31]), _i32([1] * 4)
    parents = _i32([[1, 1], [0, 0]])
    plans, copies = [], []

    def step():
        plans.append(fp4.kv_pages_extend(pool, table, lens, one, 4))
        copies.append(fp4.kv_pages_reorder(table, lens, parents, 16))
        fp4.kv_pages_collect(pool, table, lens)

    call = fp4.prepare(step)
    want = [15, 15, 31, 31]
    for _ in range(3):
        call()
        want, slots, positions, cu_q, cu_k = host.extend(want, [1] * 4, 4)
        recs = []
        for b, p in ((0, [1, 1]), (2, [0, 0])):
            rows, rec = _reorder_host(host.table[b:b + 2], want[b:b + 2], p, 16)
            host.table[b:b + 2] = rows
            recs += rec
        host.collect(want)
        assert plans[0].slots.tolist() == slots and lens.tolist() == want and copies[0].tolist() == recs
        _equal(host, pool, table, "replay")


def test_two_plans_of_one_pool_in_a_row():
    """Calls in order on one stream see each other's pages, without a wait between them."""
    fp4 = _fp4()
    host, pool, table, _ = _start(fp4, 6, 9, 16, 50, [0] * 6, 9)
    lens, dl = [0] * 6, _i32([0] * 6)
    plans = [fp4.kv_pages_extend(pool, table, dl, _i32([i, 3, 0, 7 * i, 20, 1]), 24 + 8 * i) for i in range(6)]
    for i, plan in enumerate(plans):
        lens, slots, positions, cu_q, cu_k = host.extend(lens, [i, 3, 0, 7 * i, 20, 1], 24 + 8 * i)
        assert (plan.slots.tolist(), plan.positions.tolist(), plan.cu_q.tolist(), plan.cu_k.tolist()) == (slots, positions, cu_q, cu_k), i
    _equal(host, pool, table, "all")


@pytest.mark.parametrize("seqs", [300, 5000])
def test_extend_among_empty_sequences(seqs):
    """Few sequences take tokens, far apart and next to each other, in both forms of the call."""
    fp4 = _fp4()
    for counts in ({0: 3, 70: 1, 71: 200, 131: 64, 299: 65}, {299: 1}, {0: 1}, {64: 63, 128: 1, 192: 64}, {5: 3000, 290: 1}):
        lens, new = [7] * seqs, [0] * seqs
        for b, n in counts.items():
            new[b + (seqs - 300) if b > 200 else b] = n
        host, pool, table, _ = _start(fp4, seqs, 200, 16, seqs + 220, lens, 1)
        dl, tokens = _i32(lens), sum(new) + 2
        plan = fp4.kv_pages_extend(pool, table, dl, _i32(new), tokens)
        lens, slots, positions, cu_q, cu_k = host.extend(lens, new, tokens)
        assert (dl.tolist(), plan.slots.tolist(), plan.positions.tolist()) == (lens, slots, positions)
        assert (plan.cu_q.tolist(), plan.cu_k.tolist()) == (cu_q, cu_k)
        _equal(host, pool, table, counts)


def test_a_refusal_holds_back_the_pages_behind_it():
    """After a sequence that the pool cannot serve, all later ones that need a page are refused too, whatever is free; what
    needs none is served, and a sequence refused for another reason holds nothing back."""
    fp4 = _fp4()
    for first, given in ((96, [False, False, True, True]), (129, [False, True, True, True]), (80, [True, False, True, True])):
        pool = fp4.KVPages(_i32([10, 11, 12, 13, 14] + [-1] * 15), _i32([5, 0]), 16)
        table = _i32([[-1] * 8, [0] + [-1] * 7, [1] + [-1] * 7, [2] + [-1] * 7])
        lens, new = [0, 16, 3, 15], [first, 1, 13, 1]
        dl = _i32(lens)
        plan = fp4.kv_pages_extend(pool, table, dl, _i32(new), sum(new))
        assert dl.tolist() == [a + b if g else a for a, b, g in zip(lens, new, given)], first
        assert pool.state.tolist() == [5 - 5 * given[0] - given[1], given.count(False)]
        slots = plan.slots.tolist()
        assert (min(slots[:first]) >= 0) == given[0] and (slots[first] >= 0) == given[1] and min(slots[first + 1:]) >= 16


def test_collect_over_all_holders():
    """A pool that serves two batches' tables and a kept prompt: one table that holds the rows of all of them is collected."""
    fp4 = _fp4()
    pages, page, width = 40, 16, 6
    pool = fp4.KVPages.alloc(pages, page)
    rows = torch.full((7, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(7, dtype=torch.int32, device="cuda")
    parts = [slice(0, 3), slice(3, 6), slice(6, 7)]  # views of one table: two batches and the prompt
    for part, new in zip(parts, ([20, 1, 60], [16, 33, 5], [48])):
        fp4.kv_pages_extend(pool, rows[part], lens[part], _i32(new), sum(new))
    held = {p for r, n in zip(rows.tolist(), lens.tolist()) for p in r[:-(-n // page)]}
    assert len(held) == pages - int(pool.state[0]) == 2 + 1 + 4 + 1 + 3 + 1 + 3
    lens[4] = 0  # one sequence of the second batch ends
    back = set(rows[4, :3].tolist())
    fp4.kv_pages_collect(pool, rows, lens)
    assert set(pool.free[:int(pool.state[0])].tolist()) == set(range(pages)) - held | back
    before = rows.clone()
    plan = fp4.kv_pages_extend(pool, rows[parts[0]], lens[parts[0]], _i32([16, 16, 16]), 48)
    got = {s // page for s in plan.slots.tolist()}
    kept = {p for r, n in zip(before.tolist()[3:], lens.tolist()[3:]) for p in r[:-(-n // page)]}
    assert not got & kept
