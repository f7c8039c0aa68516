"""Pages for new tokens where tables and pools end (cfz_kv8_reserve): equal to the model (oracle/pages.py)."""
import numpy as np
import pytest
import torch

from test_gpu_kv8_pages import DEV, _need_gpu, both, check, empty, ints  # noqa: F401

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
