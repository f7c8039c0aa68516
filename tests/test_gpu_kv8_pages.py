"""The pages of the 8-bit cache: free, fork, reserve, compact and copy against their model
(oracle/pages.py), equal to the last integer and byte; and a run of them with the cache's other calls
against the same tokens held densely."""
import numpy as np
import pytest
import torch

from oracle import pages as model

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_activation_residual_amd import cfz, kv8
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def both(table, lengths, refs, page):
    return (kv8.Pages(ints(table), ints(lengths), ints(refs), page),
            model.Pages(table, lengths, refs, page))


def empty(pages, batch, width, page=32):
    return both(np.full((batch, width), -1), np.zeros(batch, int), np.zeros(pages, int), page)


def check(p, m):
    assert p.table.tolist() == m.table
    assert p.lengths.tolist() == m.lengths
    assert p.refs.tolist() == m.refs


def reserve(p, m, counts, max_new, grow=True):
    moves, missing = p.reserve(ints(counts), max_new)
    source, target, lack = m.reserve(list(counts), max_new)
    assert (moves.source.tolist(), moves.target.tolist(), missing.tolist()) == (source, target, [lack])
    check(p, m)
    if grow and not lack:
        add = np.clip(counts, 0, max_new)
        p.lengths += ints(add)
        m.lengths = [a + int(b) for a, b in zip(m.lengths, add)]
    return lack


def compact(p, m):
    moves, live = p.compact()
    want, n = m.compact()
    k = int(moves.count)
    assert (int(live), k) == (n, len(want))
    assert list(zip(moves.source[:k].tolist(), moves.target[:k].tolist())) == want
    check(p, m)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("page,pages,batch,width", [(32, 60, 7, 9), (64, 5000, 40, 30),
                                                    (128, 40000, 300, 70)])
def test_runs_of_calls(seed, page, pages, batch, width):
    rng = np.random.default_rng([seed, page])
    p, m = empty(pages, batch, width, page)
    for step in range(12):
        n = int(rng.integers(1, batch + 1))
        longest = int(rng.choice([1, 2, page, page + 1, 5 * page]))
        room = np.maximum(0, width * page - np.array(m.lengths))
        counts = np.minimum(rng.integers(-1, longest + 1, batch), room) * (rng.random(batch) < 0.7)
        if reserve(p, m, counts, longest):
            p.free(ints(np.arange(batch // 2)))
            m.free(list(range(batch // 2)))
            check(p, m)
        a, c = rng.integers(-1, batch + 1, (2, n))
        p.fork(ints(a), ints(c))
        m.fork(list(map(int, a)), list(map(int, c)))
        check(p, m)
        rows = rng.integers(-1, batch + 1, n // 3 + 1)
        keep = rng.integers(-3, 4 * page, len(rows))
        p.free(ints(rows), ints(keep))
        m.free(list(map(int, rows)), list(map(int, keep)))
        check(p, m)
        named = [q for row in m.table for q in row if q >= 0]
        assert np.array_equal(np.bincount(named, minlength=pages), m.refs)
        if step % 4 == 3:
            compact(p, m)


def test_every_holder_writes():
    """All holders of a page write: the first keeps it.  Some do: each gets a copy.  At a page's border
    nothing is copied."""
    p, m = empty(20, 6, 4)
    reserve(p, m, [40, 64, 0, 0, 0, 0], 64)
    for a, c in (([0, 0], [2, 3]), ([1], [4])):
        p.fork(ints(a), ints(c))
        m.fork(a, c)
        check(p, m)
    saved = p.table.clone(), p.lengths.clone(), p.refs.clone()
    assert reserve(p, m, [1, 1, 1, 1, 1, 0], 1) == 0
    assert p.refs[saved[0][0, 1].item()] == 1 and p.table[0, 1] == saved[0][0, 1]
    # rows 2 and 3 alone: row 0 still reads the page
    q, n = both(*(t.tolist() for t in saved), 32)
    assert reserve(q, n, [0, 0, 1, 1, 0, 0], 1) == 0
    assert q.refs[saved[0][0, 1].item()] == 1 and q.table[0, 1] == saved[0][0, 1]
    # again without writing: nothing is given out twice
    before = q.table.clone()
    q.lengths -= ints([0, 0, 1, 1, 0, 0])
    n.lengths = q.lengths.tolist()
    reserve(q, n, [0, 0, 1, 1, 0, 0], 1, grow=False)
    assert torch.equal(before, q.table)


def test_too_few_pages_changes_nothing():
    p, m = empty(5, 3, 8)
    reserve(p, m, [96, 0, 0], 96)
    state = [t.clone() for t in (p.table, p.lengths, p.refs)]
    assert reserve(p, m, [33, 64, 1], 64) == 3
    assert all(torch.equal(a, b) for a, b in zip(state, (p.table, p.lengths, p.refs)))
    assert reserve(p, m, [32, 32, 0], 64) == 0
    assert reserve(p, m, [0, 0, 0], 0) == 0


def test_rows_past_the_end_and_no_pages():
    p, m = empty(9, 2, 3)
    reserve(p, m, [96, 200], 200)          # the second reaches past its row
    reserve(p, m, [5, 5], 5)               # both are full
    q, n = empty(0, 2, 3)
    assert reserve(q, n, [1, 0], 1) == 1
    compact(q, n)
    one, n1 = empty(1, 1, 1)
    assert reserve(one, n1, [32], 32) == 0
    compact(one, n1)


def test_numbers_out_of_range():
    """Places, lengths and counts that name nothing."""
    table = [[0, 99, -7, 3], [3, 1 << 30, 2, -1]]
    for lengths in ([100, 70], [-5, 1 << 30], [97, 0]):
        p, m = both(table, lengths, [1, 0, 1, 2, 0, 0, 0, 0], 32)
        reserve(p, m, [1 << 30, -(1 << 31)], 40, grow=False)
        p.fork(ints([0, 5]), ints([1, -2]))
        m.fork([0, 5], [1, -2])
        check(p, m)
        p.free(ints([0, 0, 7]), ints([40, 33, 1]))
        m.free([0, 0, 7], [40, 33, 1])
        check(p, m)


@pytest.mark.parametrize("pages", [2, 4095, 4096, 4097, 300001])
@pytest.mark.parametrize("part", [0.0, 0.3, 0.97, 1.0])
def test_packing(pages, part):
    rng = np.random.default_rng(pages)
    used = rng.random(pages) < part
    if part == 1.0:
        used[:] = True
    held = rng.permutation(np.flatnonzero(used))
    width = 64
    batch = max(1, -(-len(held) // width))
    table = np.full(batch * width, -1)
    table[:len(held)] = held
    refs = used.astype(int)
    p, _ = both(table.reshape(batch, width).tolist(), [0] * batch, refs.tolist(), 64)
    moves, live = p.compact()
    n, k = len(held), int(moves.count)
    low, high = np.flatnonzero(~used[:n]), np.flatnonzero(used)[::-1]
    assert (int(live), k) == (n, len(low))
    assert np.array_equal(moves.target[:k].cpu().numpy(), low)
    assert np.array_equal(moves.source[:k].cpu().numpy(), high[:len(low)])
    to = np.arange(pages)
    to[high[:len(low)]] = low
    want = np.where(table >= 0, to[table], -1)
    assert np.array_equal(p.table.cpu().numpy().reshape(-1), want)
    assert np.array_equal(p.refs.cpu().numpy(), np.arange(pages) < n)


def fill(pages, heads, dim, page, fmt, pooled, seed):
    c = kv8.Cache(pages, heads, dim, page, fmt, pooled=pooled, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    for t in buffers(c):
        t.view(torch.uint8).random_(0, 120, generator=g)
    return c


def buffers(c):
    return [t for t in (c.k, c.v, c.k_scale, c.v_scale, c.k_mean) if t is not None]


@pytest.mark.parametrize("heads,dim,page,fmt,pooled", [
    (1, 64, 32, "int8", True), (3, 128, 64, "e4m3", True), (30, 64, 128, "int8", False),
    (33, 128, 128, "int8", True), (1024, 64, 32, "e4m3", True)])
def test_copy(heads, dim, page, fmt, pooled):
    c = fill(9, heads, dim, page, fmt, pooled, 1)
    other = fill(5, heads, dim, page, fmt, True, 2)
    for origin, count in ((None, None), (other, None), (None, 2), (other, 0), (other, -4),
                          (None, 99)):
        before = [t.clone() for t in buffers(c)]
        source, target = [3, -1, 4, 0, 99, 1], [8, 5, 2, 9, 6, 7]
        moves = kv8.Moves(ints(source), ints(target), None if count is None else ints([count]))
        c.copy(moves, origin=origin)
        rows = origin or c
        for t, old, x in zip(buffers(c), before, buffers(rows)):
            want = old.clone()
            for i, (a, b) in enumerate(zip(source, target)):
                if 0 <= a < rows.pages and 0 <= b < 9 and (count is None or i < count):
                    want[b] = (old if origin is None else x)[a]
            assert torch.equal(t.view(torch.uint8), want.view(torch.uint8))
    c.copy(kv8.Moves(ints([]), ints([])))


def test_copy_refusals():
    c = fill(2, 2, 64, 32, "int8", True, 1)
    moves = kv8.Moves(ints([0]), ints([1]))
    for other in (fill(2, 1, 64, 32, "int8", True, 1), fill(2, 2, 128, 32, "int8", True, 1),
                  fill(2, 2, 64, 64, "int8", True, 1), fill(2, 2, 64, 32, "e4m3", True, 1),
                  fill(2, 2, 64, 32, "int8", False, 1)):
        with pytest.raises(cfz.CfzError):
            c.copy(moves, origin=other)
    for bad in (kv8.Moves(ints([0]), ints([0, 1])), kv8.Moves(ints([0]), ints([1]), ints([1, 1])),
                kv8.Moves(ints([0]), ints([1]).cpu())):
        with pytest.raises(ValueError):
            c.copy(bad)
    with pytest.raises(TypeError):
        c.copy(kv8.Moves(ints([0]).long(), ints([1])))


def test_copies_past_4_gib():
    """Pages whose bytes lie past 2^32."""
    c = kv8.Cache(530000, 4, 64, 32, "int8", pooled=False, device=DEV)
    c.k[3], c.v[3], c.k_scale[3], c.v_scale[3] = 5, 7, 0.5, 0.25
    c.copy(kv8.Moves(ints([3]), ints([529999])))
    c.copy(kv8.Moves(ints([529999]), ints([9])))
    for at in (529999, 9):
        assert (c.k[at] == 5).all() and (c.v[at] == 7).all()
        assert (c.k_scale[at] == 0.5).all() and (c.v_scale[at] == 0.25).all()
    assert not c.k[8].any() and not c.k[10].any() and not c.k[529998].any()


# ------------------------------------------------------------------ a run of them, as they are used

def test_beams_share_and_part():
    """Prompts, forks, single tokens on every branch, branches dropped and replaced, the pool packed: at
    each step the attention equals that over a cache of its own for every row, bit for bit, where
    the branches' pages were coded by the same calls."""
    heads, dim, page, batch, width = 2, 64, 32, 6, 8
    g = torch.Generator().manual_seed(1)

    def rows(n, h=heads):
        return torch.randn((n, h, dim), generator=g).bfloat16().to(DEV)

    cache = kv8.Cache(40, heads, dim, page, device=DEV)
    second = kv8.Cache(40, heads, dim, page, "e4m3", device=DEV)  # another layer, the same pages
    pages = kv8.Pages.empty(40, batch, width, page, DEV)
    plain = kv8.Cache(batch * width, heads, dim, page, device=DEV)
    own = ints(np.arange(batch * width).reshape(batch, width))
    held = [0] * batch

    def put(counts, k, v):
        offsets = ints(np.concatenate([[0], np.cumsum(counts)]))
        moves, missing = pages.reserve(ints(counts), max(counts))
        assert int(missing) == 0
        for c in (cache, second):
            c.copy(moves)
            c.append(k, v, pages.table, pages.lengths, offsets, max(counts))
        plain.append(k, v, own, ints(held), offsets, max(counts))
        pages.lengths += ints(counts)
        held[:] = [a + b for a, b in zip(held, counts)]

    def same():
        q = rows(batch, 4)
        one = ints(range(batch + 1))
        a, la = cache.attend(q, pages.table, pages.lengths, one, 1, 8 * page)
        b, lb = plain.attend(q, own, ints(held), one, 1, 8 * page)
        assert torch.equal(a, b) and torch.equal(la, lb)
        assert pages.lengths.tolist() == held

    def fork(a, c):
        pages.fork(ints(a), ints(c))
        for x, y in zip(a, c):
            plain.copy(kv8.Moves(own[x].clone(), own[y].clone()))
            held[y] = held[x]

    put([70, 64, 0, 0, 0, 33], rows(167), rows(167))
    same()
    fork([0, 0, 1], [2, 3, 4])
    same()
    for _ in range(3):
        put([1] * batch, rows(batch), rows(batch))
        same()
    fork([2, 2], [0, 3])
    pages.free(ints([5]))
    held[5] = 0
    same()
    put([40, 1, 0, 2, 3, 50], rows(96), rows(96))
    same()
    before = second.gather(pages.table, pages.lengths * 0, ints([0, held[3]] + [held[3]] * 5)
                           , held[3], held[3])
    moves, live = pages.compact()
    for c in (cache, second):
        c.copy(moves)
    same()
    after = second.gather(pages.table, pages.lengths * 0, ints([0, held[3]] + [held[3]] * 5)
                          , held[3], held[3])
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    n = int(live)
    assert n < 40 and (pages.refs[:n] > 0).all() and not pages.refs[n:].any()
    # the packed front is a cache of its own (checkpoint)
    front = kv8.Cache.over(*(t[:n].clone() for t in buffers(cache)))
    q, one = rows(batch, 4), ints(range(batch + 1))
    a, _ = front.attend(q, pages.table, pages.lengths, one, 1, 8 * page)
    b, _ = cache.attend(q, pages.table, pages.lengths, one, 1, 8 * page)
    assert torch.equal(a, b)


def test_captured_step_replays():
    """Drop, fork, reserve and copy recorded once, replayed on new lists."""
    cache = fill(64, 2, 64, 32, "int8", True, 3)
    p, m = empty(64, 8, 6)
    p.reserve(ints([50] * 4 + [0] * 4), 50)
    m.reserve([50] * 4 + [0] * 4, 50)
    p.lengths += ints([50] * 4 + [0] * 4)
    m.lengths = p.lengths.tolist()
    rows, parents, counts = ints([4, 5]), ints([0, 0]), ints([1] * 8)

    def step():
        p.free(rows)
        p.fork(parents, rows)
        moves, missing = p.reserve(counts, 1)
        cache.copy(moves)
        return moves, missing

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        saved = [t.clone() for t in (p.table, p.lengths, p.refs)]
        step()
        for t, s in zip((p.table, p.lengths, p.refs), saved):
            t.copy_(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moves, missing = step()
    for a, c in (([0, 0], [4, 5]), ([1, 4], [6, 5]), ([3, 3], [7, 7])):
        rows.copy_(ints(c))
        parents.copy_(ints(a))
        graph.replay()
        torch.cuda.synchronize()
        m.free(c)
        m.fork(a, c)
        assert (moves.source.tolist(), moves.target.tolist(), missing.tolist()) == \
            tuple(x if isinstance(x, list) else [x] for x in m.reserve([1] * 8, 1))
        check(p, m)
        for s, t in zip(moves.source.tolist(), moves.target.tolist()):
            if s >= 0:
                assert torch.equal(cache.k[s], cache.k[t]) and torch.equal(cache.k_mean[s],
                                                                          cache.k_mean[t])


def test_refusals_of_the_binding():
    p, _ = empty(8, 2, 4)
    rows = ints([0])
    for call in (lambda: p.free(rows.long()), lambda: p.free(rows.cpu()), lambda: p.free(rows[None]),
                 lambda: p.free(rows, ints([1, 2])), lambda: p.fork(rows, ints([0, 1])),
                 lambda: p.fork(rows.long(), rows), lambda: p.reserve(ints([1]), 1),
                 lambda: p.reserve(ints([1, 1]), -1), lambda: p.reserve(ints([1, 1]), 1 << 64),
                 lambda: p.reserve(ints([1, 1]), 1, workspace=torch.empty(8, device=DEV)),
                 lambda: p.compact(workspace=torch.empty(4, device=DEV)),
                 lambda: p.compact(workspace=torch.empty(4096)),
                 lambda: kv8.Pages(p.table.cpu(), p.lengths, p.refs, 32),
                 lambda: kv8.Pages(p.table[0], p.lengths, p.refs, 32),
                 lambda: kv8.Pages(p.table, p.lengths[:1], p.refs, 32),
                 lambda: kv8.Pages(p.table, p.lengths, p.refs.long(), 32),
                 lambda: kv8.Pages(p.table.t(), p.lengths, p.refs, 32),
                 lambda: kv8.Pages(p.table, p.lengths, p.refs, 48).free(rows)):
        with pytest.raises((ValueError, TypeError, cfz.CfzError)):
            call()
    assert (p.table == -1).all() and not p.lengths.any() and not p.refs.any()
