"""Pages for new tokens where tables and pools end (cfz_kv8_reserve): equal to the model (oracle/pages.py)."""
import itertools
import threading

import numpy as np
import pytest
import torch

from test_gpu_kv8_pages import DEV, _need_gpu, both, check, compact, empty, ints  # noqa: F401

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_activation_residual_amd import kv8


def reserve(p, m, counts, max_new):
    want = m.left_out(list(map(int, counts)), max_new)
    moves, missing = p.reserve(ints(counts), max_new)
    source, target, lack = m.reserve(list(map(int, counts)), max_new)
    assert moves.left_out.tolist() == want
    assert (moves.source.tolist(), moves.target.tolist(), missing.tolist()) == (source, target, [lack])
    check(p, m)
    return moves, lack


def test_rows_that_are_full_say_so():
    """A caller who goes on by what has a place loses no token without knowing of it."""
    p, m = empty(12, 4, 3)
    total = np.zeros(4, int)
    for counts in ([96, 90, 0, 33], [1, 6, 5, 63], [0, 7, 200, 1], [3, -4, 0, 0]):
        moves, lack = reserve(p, m, counts, 200)
        assert lack == 0
        p.lengths += ints(np.maximum(counts, 0)) - moves.left_out
        m.lengths = [min(n + max(0, c), 96) for n, c in zip(m.lengths, counts)]
        check(p, m)
        total += np.maximum(counts, 0)
    assert p.lengths.tolist() == np.minimum(total, 96).tolist()


def test_left_out_counts_what_exceeds_a_call_too():
    p, m = empty(3, 5, 2)
    reserve(p, m, [40, 7, 8, 1 << 30, -(1 << 31)], 7)          # more than max_new
    m.lengths = [64, 70, -5, 63, 1 << 30]
    p.lengths.copy_(ints(m.lengths))
    reserve(p, m, [1, 1, 70, 2, (1 << 31) - 1], (1 << 31) - 1)  # lengths past the table, and below 0
    moves, lack = reserve(p, m, [0, 0, 64, 64, 0], 64)          # too few pages: what is full is said all the same
    q, n = empty(2, 2, 4)
    moves, lack = reserve(q, n, [200, 130], 200)
    assert lack == 6 and moves.left_out.tolist() == [72, 2]


@pytest.mark.parametrize("seed", range(4))
def test_left_out_of_many_rows(seed):
    rng = np.random.default_rng(seed)
    p, m = empty(3000, 2500, 3)
    m.lengths = [int(n) for n in rng.integers(-3, 110, 2500)]
    p.lengths.copy_(ints(m.lengths))
    reserve(p, m, rng.integers(-2, 60, 2500), int(rng.integers(0, 80)))


def crowded(pages, free, batch, width, rng, page=32):
    """Rows that hold every page but the free ones, in any order; the last rows are empty."""
    used = np.setdiff1d(np.arange(pages), free)
    table = np.full((batch, width), -1)
    table.reshape(-1)[:len(used)] = rng.permutation(used)
    refs = np.zeros(pages, int)
    refs[used] = 1
    return both(table, (table >= 0).sum(1) * page, refs, page)


@pytest.mark.parametrize("need", [1, 1023, 1024, 1025, 2049, 3000])
def test_free_pages_behind_many_in_use(need):
    """Free pages on either side of every 16,384 looked at, and more of them than the chip keeps."""
    rng = np.random.default_rng(need)
    around = np.concatenate([np.arange(k - 3, k + 3) for k in (16384, 32768, 49152)])
    free = np.concatenate([[5], around, np.sort(rng.choice(np.arange(49200, 56000), need, False))])
    p, m = crowded(56000, free, 900, 70, rng)
    assert m.lengths[805:] == [0] * 95
    counts = np.zeros(900, int)
    pages = need + 5  # (some of the last ones stay free)
    for row in range(810, 900):
        counts[row] = 32 * min(pages, 70) - int(rng.integers(0, 32) if pages > 1 else 0)
        pages -= min(pages, 70)
    assert pages == 0
    _, lack = reserve(p, m, counts, 70 * 32)
    assert lack == 0
    # what is left is not enough: nothing changes, after looking through all of them
    again = np.zeros(900, int)
    again[805:810] = 70 * 32
    _, lack = reserve(p, m, again, 70 * 32)
    assert lack == 5 * 70 - (len(free) - need - 5)


def test_many_copies_of_shared_pages():
    """More than 1024 rows about to write into pages that others hold; the new pages come through memory."""
    rng = np.random.default_rng(7)
    p, m = crowded(20000, np.arange(100, 20000, 5), 6000, 4, rng)
    lengths = [max(0, n - int(k)) for n, k in zip(m.lengths, rng.integers(1, 32, 6000))]
    m.lengths = lengths
    p.lengths.copy_(ints(lengths))
    first = next(i for i in range(6000) if m.table[i][0] < 0)
    children = np.arange(first, 6000)
    parents = rng.integers(0, 900, len(children))
    p.fork(ints(parents), ints(children))
    m.fork(list(map(int, parents)), list(map(int, children)))
    check(p, m)
    moves, lack = reserve(p, m, np.ones(6000, int), 1)
    assert lack == 0 and (moves.source >= 0).sum() > 1024
    p.free(ints(children))
    m.free(list(map(int, children)))
    check(p, m)


def test_beside_a_thread_that_allocates():
    """Another thread takes and fills blocks of the workspaces' sizes on the same stream all the while."""
    p, m = empty(600, 200, 4)
    stop = threading.Event()

    def busy():
        for size in itertools.cycle((4 * (2 * 200 + 2 * 600), 4 * 601, 4 * 601, 256)):
            if stop.is_set():
                return
            torch.empty(size, dtype=torch.uint8, device=DEV).fill_(255)

    other = threading.Thread(target=busy)
    other.start()
    try:
        rng = np.random.default_rng(1)
        for step in range(60):
            counts = rng.integers(0, 2, 200)
            _, lack = reserve(p, m, counts, 1)
            p.lengths += ints(counts) * (lack == 0)
            m.lengths = [a + int(b) * (lack == 0) for a, b in zip(m.lengths, counts)]
            gone = [int(i) for i in rng.integers(0, 200, 6)]
            p.free(ints(gone))
            m.free(gone)
            compact(p, m)
    finally:
        stop.set()
        other.join()
    check(p, m)
