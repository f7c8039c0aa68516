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
