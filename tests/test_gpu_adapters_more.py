"""The adapters where their rows are left alone to the last bit, and in every tile of the first product
(test_gpu_adapters.py has the ranks, slices and refusals)."""
import numpy as np
import pytest
import torch

from test_gpu_adapters import DEV, REAL, check, make  # noqa: F401
from test_gpu_block import Gen, _need_gpu, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("real", ["bf16", "f16"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("slices", [[16], [48, 320]])
def test_rows_without_an_adapter_keep_every_bit(real, wide, slices):
    """Any bits: zeros of either sign, infinities, NaNs of any kind."""
    g = Gen(41)
    w = make(g, 1, 64, slices, 8, real)
    counts = [70, 1, 16, 33]
    off, ids = np.concatenate([[0], np.cumsum(counts)]), [-1, 0, 7, -(1 << 31)]
    n, cols = int(off[-1]), sum(slices)
    like = torch.int32 if wide else torch.int16
    bits = torch.randint(-(1 << 15), 1 << 15, (n, cols), generator=g.g)
    if wide:
        bits = bits << 16 | torch.randint(0, 1 << 16, (n, cols), generator=g.g)
    bits = bits.to(like).to(DEV)
    bits[:, ::3] = torch.iinfo(like).min  # -0
    y = bits.view(torch.float32 if wide else REAL[real])
    x = g(n, 64, dtype=REAL[real])
    out = w.add(x, y, ints(ids), ints(off), 70)
    away = np.ones(n, bool)
    away[off[1]:off[2]] = False
    away = torch.tensor(away, device=DEV)
    assert torch.equal(out.view(like)[away], bits[away])
    held = y.clone()
    w.add(x, held, ints(ids), ints(off), 70, out=held)
    assert torch.equal(held.view(like), out.view(like))


def ragged(tokens, batch, rng):
    """Lengths of tokens in all, one sequence empty, ends off the tiles' borders."""
    cuts = np.sort(rng.choice(np.arange(1, tokens), batch - 2, False))
    return [int(n) for n in np.concatenate([[0], cuts, cuts[-1:], [tokens]])]


def run(seed, tokens, batch, cols_in, slices, rank, real, wide=False):
    rng, g = np.random.default_rng([seed, tokens, cols_in]), Gen(seed)
    w = make(g, 4, cols_in, slices, rank, real)
    off = ragged(tokens, batch, rng)
    ids = [int(i) for i in rng.integers(-1, 5, batch)]
    ids[0] = 2
    x = g(tokens, cols_in, dtype=REAL[real])
    y = g(tokens, sum(slices), dtype=torch.float32 if wide else REAL[real])
    out = w.add(x, y, ints(ids), ints(off), tokens)
    check(w, x, y, out, ids, off, real)


@pytest.mark.parametrize("real", ["bf16", "f16"])
@pytest.mark.parametrize("slices,rank", [([16], 8), ([16, 32, 16], 8), ([32], 24), ([16, 48], 24),
                                         ([64], 64), ([16, 16], 40), ([16, 32, 16], 32), ([16], 96),
                                         ([16, 16, 16, 16], 24)])
def test_tiles_of_64_tokens(real, slices, rank):
    """Sequences long enough for 128 tiles of 64 tokens, up to 96 adapter rows; columns that leave waves
    without any, and that end inside a step."""
    for cols_in in (8, 136, 1000, 1928):
        run(rank, 8300, 5, cols_in, slices, rank, real)


@pytest.mark.parametrize("real", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,batch,slices,rank", [
    (8191, 3, [16], 32), (8192, 3, [16], 32),      # 127 whole tiles of 64 tokens, and 128
    (8256, 130, [16], 32), (8320, 130, [16], 32),  # 63 and 64 tokens a sequence
    (4095, 64, [16], 32), (4096, 64, [16], 32),
    (8300, 3, [16, 16], 48), (8300, 3, [16], 104), (8300, 3, [16], 128), (8300, 3, [16, 16], 72),
    (500, 16, [16], 64), (512, 16, [16], 64), (300, 3, [16, 16], 64), (300, 3, [16, 16, 16], 48)])
def test_either_side_of_the_tiles_thresholds(real, tokens, batch, slices, rank):
    run(tokens, tokens, batch, 264, slices, rank, real, wide=real == "bf16")


@pytest.mark.parametrize("real", ["bf16", "f16"])
def test_a_prompt_beside_single_tokens(real):
    g = Gen(51)
    w = make(g, 3, 520, [32, 16], 16, real)
    counts = [1] * 40 + [700] + [1] * 30
    off = [int(n) for n in np.concatenate([[0], np.cumsum(counts)])]
    ids = [i % 5 - 1 for i in range(len(counts))]
    ids[40] = 1
    x, y = g(off[-1], 520, dtype=REAL[real]), g(off[-1], 48, dtype=REAL[real])
    check(w, x, y, w.add(x, y, ints(ids), ints(off), 700), ids, off, real)
