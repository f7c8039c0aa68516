"""GPU parity of the low-rank adapters beside a shared projection against their 64-bit model
(oracle/block.py), within the model's bound and one rounding of the result."""
import numpy as np
import pytest
import torch

from oracle import block as model
from test_gpu_block import REAL, Gen, _need_gpu, close, ints, to64  # noqa: F401

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_activation_residual_amd import block, cfz
DEV = "cuda:0"


def make(g, count, cols_in, slices, rank, real, scaled=True):
    a = g(count, len(slices) * rank, cols_in, dtype=REAL[real], size=cols_in ** -0.5)
    b = g(count, sum(slices), rank, dtype=REAL[real], size=rank ** -0.5)
    scale = g(count) if scaled else None
    w = block.Adapters(a, b, scale, slices=slices)
    w.rows = a
    return w


def check(w, x, y, out, ids, offsets, real, before=None, max_rows=1 << 30):
    seen = np.zeros(len(y), bool)
    for i, n in enumerate(ids):
        lo, hi = offsets[i], min(offsets[i + 1], offsets[i] + max_rows)
        if lo >= hi:
            continue
        seen[lo:hi] = True
        if not 0 <= n < w.count:
            assert torch.equal(out[lo:hi], y[lo:hi])
            continue
        want, off = model.adapters_add(to64(x[lo:hi]), to64(y[lo:hi]), to64(w.rows[n]), to64(w.b[n]),
                                       1.0 if w.scale is None else float(w.scale[n]), w.slices, real)
        close(out[lo:hi], want, off)
    if before is not None:
        assert (to64(out)[~seen] == before).all()


@pytest.mark.parametrize("real", ["bf16", "f16"])
@pytest.mark.parametrize("rank,slices,cols_in", [
    (8, [16], 8), (8, [48, 16, 16], 72), (16, [64], 64), (24, [80, 208], 520), (32, [256], 1024),
    (40, [1024, 128, 128], 512), (64, [512], 4096), (64, [64, 64, 64, 64], 136), (128, [320], 1928),
    (128, [96, 160], 256), (104, [16, 1040], 640), (88, [64, 32, 80], 264), (128, [32, 64, 16, 48], 192),
    (72, [80, 16, 16, 16], 96), (120, [16, 48, 32], 136)])
@pytest.mark.parametrize("tall", [False, True])
def test_ranks_and_slices(real, rank, slices, cols_in, tall):
    """Every number of adapter rows, column groups that end inside a wave's, odd numbers of tokens: single
    ones and runs beside each other, sequences with one adapter, another, none, and none that exists."""
    g = Gen(rank + cols_in)
    counts = [150, 1, 0, 33, 64, 17] if tall else [1, 1, 1, 2, 0, 1, 5]
    ids = [2, 0, 1, -1, 0, 2, 99][:len(counts)]
    offsets = [3] + [3 + int(n) for n in np.cumsum(counts)]
    tokens = offsets[-1] + 2
    w = make(g, 3, cols_in, slices, rank, real)
    x = g(tokens, cols_in, dtype=REAL[real])
    y = g(tokens, sum(slices), dtype=REAL[real])
    out = torch.full_like(y, 7.0)
    got = w.add(x, y, ints(ids), ints(offsets), max(counts), out=out)
    assert got is out
    check(w, x, y, out, ids, offsets, real, before=7.0)
    again = y.clone()
    w.add(x, again, ints(ids), ints(offsets), max(counts), out=again)
    rows = slice(offsets[0], offsets[-1])
    assert torch.equal(again[rows], out[rows])
    assert torch.equal(again[:3], y[:3]) and torch.equal(again[-2:], y[-2:])


@pytest.mark.parametrize("real", ["bf16", "f16"])
def test_strides_fp32_rows_and_no_scale(real):
    g = Gen(4)
    w = make(g, 2, 256, [128, 64], 16, real, scaled=False)
    x = g(40, 512, dtype=REAL[real])[:, 256:]
    y = g(40, 200)[:, :192]
    got = w.add(x, y, ints([1, 0]), ints([0, 21, 40]), 40)
    assert got.dtype == torch.float32
    check(w, x, y, got, [1, 0], [0, 21, 40], real)
    cut = torch.full((40, 192), 7.0, device=DEV)
    w.add(x, y, ints([1, 0]), ints([0, 21, 40]), 9, out=cut)
    check(w, x, y, cut, [1, 0], [0, 21, 40], real, before=7.0, max_rows=9)


@pytest.mark.parametrize("batch", [1, 64, 65, 700, 5000])
def test_many_sequences(batch):
    """Tiles find their sequences among many, empty ones between them."""
    g = Gen(batch)
    rng = np.random.default_rng(batch)
    counts = rng.integers(0, 4, batch)
    counts[batch // 2] = 70
    offsets = np.concatenate([[0], np.cumsum(counts)])
    ids = rng.integers(-1, 6, batch)
    tokens = int(offsets[-1])
    w = make(g, 6, 64, [32], 8, "bf16")
    x, y = g(tokens, 64, dtype=torch.bfloat16), g(tokens, 32, dtype=torch.bfloat16)
    out = w.add(x, y, ints(ids), ints(offsets), 70)
    which = torch.tensor(np.repeat(ids, counts), device=DEV)
    low = torch.zeros(tokens, 32, dtype=torch.float64, device=DEV)
    for n in range(6):
        h = (x.double() @ w.rows[n].double().t().contiguous()) * w.scale[n].double()
        low += torch.where((which == n)[:, None], h @ w.b[n].double().t().contiguous(), 0.0)
    want = y.double() + low
    # (rank 8, sizes of 1: far inside the model's bound at 2^-12)
    assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -12).all()


def test_values_at_the_types_ends():
    """fp16 rows whose products pass fp16's range on the way; rows that are not finite stay alone."""
    g = Gen(8)
    w = make(g, 1, 128, [64], 16, "f16")
    x = g(9, 128, dtype=torch.float16)
    x[0] *= 15000
    x[1] = 60000
    x[2] = 2.0 ** -24
    x[3] = 0
    x[4, 5], x[5, 1] = float("nan"), float("inf")
    y = torch.zeros(9, 64, device=DEV)
    out = w.add(x, y, ints([0]), ints([0, 9]), 9)
    for rows in (slice(0, 4), slice(6, 9)):
        check(w, x[rows], y[rows], out[rows], [0], [0, rows.stop - rows.start], "f16")
    assert out[4].isnan().all() and not out[5].isfinite().any()
    # exactly zero where the adapter is
    w.b.zero_()
    assert torch.equal(w.add(x[:4], y[:4] + 3, ints([0]), ints([0, 4]), 4), y[:4] + 3)


@pytest.mark.parametrize("real", ["bf16", "f16"])
@pytest.mark.parametrize("power", [-100, -60, 60, 100])
def test_scales_of_any_size(real, power):
    """h far outside of fp16's range either way; rows that it leaves in fp32's range are right."""
    g = Gen(power + 200)
    w = make(g, 1, 64, [64], 8, real)
    w.scale.fill_(2.0 ** power)
    x, y = g(20, 64, dtype=REAL[real]), torch.zeros(20, 64, device=DEV)
    out = w.add(x, y, ints([0]), ints([0, 20]), 20)
    check(w, x, y, out, [0], [0, 20], real)
    assert out.any() and out.isfinite().all()


def test_nothing_to_add():
    g = Gen(9)
    w = make(g, 2, 64, [64], 8, "bf16")
    x, y = g(4, 64, dtype=torch.bfloat16), g(4, 64, dtype=torch.bfloat16)
    assert torch.equal(w.add(x, y, ints([-1]), ints([0, 4]), 4), y)
    assert w.add(x[:0], y[:0], ints([0]), ints([0, 0]), 4).shape == (0, 64)
    assert torch.equal(w.add(x, y, ints([]), ints([0]), 4, out=y.clone()), y)


def test_refusals():
    g = Gen(10)
    w = make(g, 2, 64, [64], 8, "bf16")
    x, y = g(4, 64, dtype=torch.bfloat16), g(4, 64, dtype=torch.bfloat16)
    one, off = ints([0]), ints([0, 4])
    for args in ((x.half(), y), (x, y.half())):
        with pytest.raises(TypeError):
            w.add(*args, one, off, 4)
    for args in ((x[:, :32], y), (x, y[:3]), (x[0], y[0])):
        with pytest.raises(ValueError):
            w.add(*args, one, off, 4)
    with pytest.raises(TypeError):
        w.add(x, y, one.long(), off, 4)
    with pytest.raises(ValueError):
        w.add(x, y, one, ints([0, 1, 4]), 4)
    with pytest.raises(cfz.CfzError):
        w.add(x, y, one, off, 4, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(cfz.CfzError):
        w.add(x, y, one, off, -1)
    for a, b, kw in ((w.rows, w.b, dict(slices=3)), (w.rows, w.b[:1], {}),
                     (w.rows[:, :4], w.b, {}), (w.rows, w.b.half(), {}),
                     (w.rows, w.b, dict(scale=y[0])), (w.rows[0], w.b, {})):
        with pytest.raises(ValueError):
            block.Adapters(a, b, **kw)
    with pytest.raises(cfz.CfzError):
        block.Adapters(w.rows[:, :4].contiguous(), w.b[:, :, :4].contiguous())
    for args in ((1, w.rows), (-1, w.rows), (0, w.rows.half()), (0, w.rows, w.b[:1]),
                 (0, w.rows, None, w.scale[:1])):
        with pytest.raises(ValueError):
            w.put(*args)


@pytest.mark.parametrize("down,cols_in", [(8, 8), (24, 40), (16, 32), (72, 4104)])
def test_layout_and_replacement(down, cols_in):
    """Pieces of 16 rows x 32 columns, zeros past the ends; adapters replaced leave the others alone."""
    g = Gen(down)
    a = g(3, down, cols_in, dtype=torch.bfloat16)
    w = block.Adapters(a, g(3, 64, down, dtype=torch.bfloat16), g(3))

    def want(rows):
        i, k = -(-down // 16), -(-cols_in // 128) * 4
        full = torch.zeros(3, 16 * i, 32 * k, dtype=torch.bfloat16, device=DEV)
        full[:, :down, :cols_in] = rows
        return full.view(3, i, 16, k, 4, 8).permute(0, 1, 3, 4, 2, 5).contiguous()

    def held():
        return w.a.view(torch.bfloat16).view(want(a).shape)

    assert torch.equal(held(), want(a))
    new, b, scale = g(2, down, cols_in, dtype=torch.bfloat16), w.b[:2].clone() + 1, g(2)
    before = w.b.clone(), w.scale.clone()
    w.put(1, new, b, scale)
    a[1:] = new
    assert torch.equal(held(), want(a))
    assert torch.equal(w.b[1:], b) and torch.equal(w.scale[1:], scale)
    assert torch.equal(w.b[0], before[0][0]) and w.scale[0] == before[1][0]
    w.put(0, a)
    assert torch.equal(held(), want(a)) and torch.equal(w.b[1:], b)


def test_streams_and_graphs():
    g = Gen(11)
    w = make(g, 3, 1024, [512, 128, 128], 16, "bf16")
    x, y = g(37, 1024, dtype=torch.bfloat16), g(37, 768, dtype=torch.bfloat16)
    ids, off = ints([2, 0, -1, 1]), ints([0, 1, 20, 21, 37])
    want = w.add(x, y, ids, off, 19)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w.add(x, y, ids, off, 19, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = w.add(x, y, ids, off, 19)
    for _ in range(3):
        x.copy_(g(37, 1024, dtype=torch.bfloat16))
        ids.copy_(ints(np.roll([2, 0, -1, 1], _)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, w.add(x, y, ids, off, 19))


def test_rows_past_four_gigabytes():
    from test_gpu_block import far_rows
    g = Gen(31)
    w = make(g, 2, 128, [64], 16, "bf16")
    near, y = g(18, 128, dtype=torch.bfloat16), g(18, 64, dtype=torch.bfloat16)
    x, z = far_rows(18, 128, torch.bfloat16), far_rows(18, 64, torch.bfloat16)
    x.copy_(near)
    z.copy_(y)
    args = (ints([1, 0]), ints([0, 3, 18]), 18)
    want = w.add(near, y, *args)
    assert torch.equal(w.add(x, z, *args, out=z), want)


def test_two_calls_at_once():
    """On two streams, each with memory of its own, over and over; equal to one after the other."""
    g = Gen(32)
    w = make(g, 3, 1920, [640, 640], 32, "bf16")
    jobs = []
    for counts in ([700, 300], [64, 1, 500, 40]):
        off = ints(np.concatenate([[0], np.cumsum(counts)]))
        n = sum(counts)
        jobs.append((g(n, 1920, dtype=torch.bfloat16), g(n, 1280, dtype=torch.bfloat16),
                     ints(np.arange(len(counts)) % 3), off, max(counts)))
    want = [w.add(*j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        got += [(i, w.add(*j, stream=s)) for i, (j, s) in enumerate(zip(jobs, streams))]
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i]) for i, t in got)
