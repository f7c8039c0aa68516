"""Norms of rows and heads whose squares vanish in fp32 or leave its range, against the 64-bit models
(oracle/block.py) within the same bounds as any others: a power of two changes no rounding."""
import numpy as np
import pytest
import torch

from oracle import block as model
from test_gpu_block import DEV, REAL, Gen, _need_gpu, check_norm, close, to64  # noqa: F401

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_activation_residual_amd import block

SIZES = [1.0, 2.0 ** -40, 2.0 ** -76, 2.0 ** -100, 1.0, 2.0 ** 66, 2.0 ** 100, 2.0 ** -90]


def sized(g, rows, cols, dtype, kinds):
    """Rows of each size in turn."""
    x = torch.randn(rows, cols, generator=g.g, dtype=torch.float64) + 0.5
    return (x * torch.tensor([kinds[i % len(kinds)] for i in range(rows)])[:, None]).to(dtype).to(DEV)


@pytest.mark.parametrize("cols", [8, 64, 72, 200, 512, 1024, 1920, 4096, 16384])
@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norms_of_rows_of_any_size(cols, real, kind):
    g = Gen(cols)
    x, y = (sized(g, 37, cols, REAL[real], SIZES) for _ in "xy")
    stream = g(37, cols, dtype=REAL[real])
    for eps in (0.0, 1e-45, 1e-38, 1e-30, 1e-6):
        kw = dict(before=block.Norm(kind, eps, g(cols, dtype=REAL[real], mean=1)))
        _, h = block.residual_norm(x, **kw)
        check_norm([0, 37], 37, x, None, None, h, kw)
        # of a block's output, beside a stream of the usual size
        kw = dict(after=block.Norm(kind, eps), gate=g(cols))
        r, _ = block.residual_norm(stream, y, **kw)
        check_norm([0, 37], 37, stream, y, r, None, kw)


@pytest.mark.parametrize("cols", [64, 1024])
@pytest.mark.parametrize("real", ["bf16", "f32"])
def test_subnormal_rows_and_the_largest_ones(cols, real):
    """(Root mean squares: a mean of subnormal numbers has fewer bits than its bound counts.)"""
    g = Gen(cols)
    # 2^-126 and below, and up to the type's end
    x = sized(g, 24, cols, torch.float64, [2.0 ** -126, 2.0 ** -124, 1.0, 2.0 ** 122])
    x = x.clamp(-2.0 ** 127, 2.0 ** 127).to(REAL[real])
    kw = dict(before=block.Norm("rms", 0.0))
    _, h = block.residual_norm(x, **kw)
    check_norm([0, 24], 24, x, None, None, h, kw)


@pytest.mark.parametrize("cols", [64, 1024])
def test_rows_without_a_norm_stay_so(cols):
    x = torch.zeros(6, cols, device=DEV)
    x[1] = 1e-30
    x[2, 3], x[3, 5], x[4] = float("nan"), float("inf"), 2.0 ** 100
    for kind, nothing in (("rms", [0, 2]), ("layer", [0, 1, 2, 4])):
        _, h = block.residual_norm(x, before=block.Norm(kind, 0.0))
        assert h[nothing].isnan().all()
        assert h[3, 5].isnan()
        if kind == "rms":
            # (1 up to the model's bound for |v| = root = 1: U of the value, 43 U of the root, 3 U of the
            # quotient and the product, and the result's rounding, U = 2^-24)
            assert (h[[1, 4]] - 1).abs().max() <= 48 * 2.0 ** -24
            assert not h[3, :5].any() and not h[3, 6:].any()


@pytest.mark.parametrize("dim", [32, 64, 128, 256])
@pytest.mark.parametrize("real", ["bf16", "f32"])
@pytest.mark.parametrize("pairs", [None, False, True])
def test_heads_of_any_size(dim, real, pairs):
    g = Gen(dim)
    tokens, heads = 5, 19
    x = sized(g, tokens * heads, dim, REAL[real], SIZES + [2.0 ** -126, 2.0 ** 122])
    x = x.view(tokens, heads, dim)
    w = g(dim, dtype=REAL[real], mean=1)
    turn = None if pairs is None else block.rotation_table(dim // 2, rows=tokens, interleaved=pairs,
                                                           device=DEV)
    cos, sin = (None, None) if turn is None else (to64(turn.cos), to64(turn.sin))
    for eps in (0.0, 1e-38, 1e-6):
        (out,) = block.rotate([x], turn, weights=[w], eps=eps)
        close(out, *model.rotate(to64(x), cos, sin, pairs, True, float(np.float32(eps)), to64(w)))
