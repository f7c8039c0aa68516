"""GPU parity of the norms around a block and of the rotation of queries and keys against their
64-bit models (oracle/block.py), within the models' bounds on fp32 arithmetic plus one rounding of
the result: half a step, eps / 2 of its size, and half the smallest subnormal."""
import numpy as np
import pytest
import torch

from oracle import block as model

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_activation_residual_amd import block, cfz, kv8
DEV = "cuda:0"
REAL = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def to64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(got, want, off):
    """Each value within its bound and the rounding of the result."""
    g, t = to64(got), got.dtype
    half = torch.finfo(t).eps / 2
    err, most = np.abs(g - want), off + half * (np.abs(want) + off) + TINY[t]
    with np.errstate(invalid="ignore"):
        bad = ~(err <= most)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), g[bad][:4],
                           want[bad][:4], np.broadcast_to(most, g.shape)[bad][:4])


class Gen:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def __call__(self, *shape, dtype=torch.float32, size=1.0, mean=0.0):
        return (torch.randn(shape, generator=self.g) * size + mean).to(dtype).to(DEV)


# ------------------------------------------------------------------ the norms around a block

def check_norm(offsets, tokens, x, y, r, h, kw, untouched=None):
    """Every item's rows against the model; other rows still hold `untouched`."""
    seen = np.zeros(tokens, bool)
    row = {k: kw.get(k) for k in ("gate", "scale", "shift")}
    for b in range(len(offsets) - 1):
        a, e = offsets[b], offsets[b + 1]
        if a >= e:
            continue
        seen[a:e] = True
        item = {k: None if t is None else to64(t if t.dim() == 1 else t[min(b, t.shape[0] - 1)])
                for k, t in row.items()}
        norms = {k: None if kw.get(k) is None else
                 dict(kind=kw[k].kind, eps=float(np.float32(kw[k].eps)), weight=to64(kw[k].weight),
                      bias=to64(kw[k].bias)) for k in ("after", "before")}
        want = model.residual_norm(to64(x[a:e]), None if y is None else to64(y[a:e]),
                                   gate_scale=float(np.float32(kw.get("gate_scale", 1.0))), **item,
                                   **norms)
        if r is not None:
            close(r[a:e], want[0], want[2])
        if h is not None:
            close(h[a:e], want[1], want[3])
    if untouched is not None:
        for t in (r, h):
            assert (to64(t)[~seen] == untouched).all()


@pytest.mark.parametrize("cols", [8, 64, 72, 128, 200, 256, 264, 512, 520, 1024, 1920, 4096, 4104, 8200, 16384])
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_widths(cols, xt, yt, kind):
    g = Gen(cols)
    rows, yt = 13, REAL[yt]
    x = g(rows, cols, dtype=REAL[xt], size=3, mean=1)
    y = g(rows, cols, dtype=yt)
    kw = dict(after=block.Norm(kind, 1e-5, g(cols, dtype=yt, mean=1)), gate=g(1, cols, dtype=yt),
              before=block.Norm(kind, 1e-6, g(cols, dtype=yt), g(cols, dtype=yt) if kind == "layer"
                                else None), scale=g(cols, dtype=yt), shift=g(cols, dtype=yt),
              gate_scale=0.6)
    r, h = block.residual_norm(x, y, **kw)
    assert r.dtype == x.dtype and h.dtype == yt
    check_norm([0, rows], rows, x, y, r, h, kw)


@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"),
                                   ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("cols,f32", [(136, False), (136, True), (40, False), (72, True),
                                      (264, False), (528, True)])
def test_norm_items_gaps_and_strides(xt, yt, cols, f32):
    """Ragged items (one empty, one of one row, rows before, between nothing and behind), rows that
    lie apart, chunks of one conditioning projection."""
    g = Gen(3)
    offsets, tokens, yt = [2, 2, 9, 10, 31], 35, REAL[yt]
    vt = torch.float32 if f32 else yt
    x = g(tokens, 2 * cols, dtype=REAL[xt])[:, cols:]
    y = g(tokens, cols + 24, dtype=yt)[:, :cols]
    shift, scale, gate = g(4, 3 * cols, dtype=vt, size=0.3).chunk(3, 1)
    kw = dict(gate=gate, scale=scale, shift=shift, before=block.Norm("layer", 1e-6))
    out = torch.full((tokens, cols + 8), 7.0, dtype=x.dtype, device=DEV)
    normed = torch.full((tokens, 2 * cols), 7.0, dtype=yt, device=DEV)
    r, h = block.residual_norm(x, y, offsets=ints(offsets), out=out[:, :cols],
                               normed=normed[:, cols:], **kw)
    check_norm(offsets, tokens, x, y, r, h, kw, untouched=7.0)
    assert (out[:, cols:] == 7).all() and (normed[:, :cols] == 7).all()


@pytest.mark.parametrize("batch", [1, 63, 64, 65, 130, 4097, 65535])
def test_norm_many_items(batch):
    """Every number of items that one, two and three rounds of the search take."""
    g = Gen(batch)
    counts = np.random.default_rng(batch).integers(0, 3, batch)
    counts[0] = counts[-1] = 0
    if batch == 1:
        counts[0] = 5
    offsets = np.concatenate([[0], np.cumsum(counts)])
    tokens = int(offsets[-1]) + 2
    x = g(tokens, 8)
    shift = g(batch, 8)
    out = torch.full((tokens, 8), 7.0, device=DEV)
    _, h = block.residual_norm(x, shift=shift, offsets=ints(offsets), normed=out)
    item = np.repeat(np.arange(batch), counts)
    want = (x[:-2] + shift[torch.tensor(item, device=DEV)])
    assert torch.equal(h[:-2], want) and (h[-2:] == 7).all()


def test_norm_equal_runs_and_broadcast():
    g = Gen(5)
    x, y = g(21, 64), g(21, 64)
    scale = g(3, 64)
    kw = dict(scale=scale, gate=g(64), before=block.Norm("rms", 0.0))
    r, h = block.residual_norm(x, y, **kw)
    check_norm([0, 7, 14, 21], 21, x, y, r, h, kw)
    with pytest.raises(cfz.CfzError):
        block.residual_norm(x[:20], y[:20], **kw)


def test_norm_parts_of_a_step():
    """The sum alone, the norm alone, in place, no rows at all."""
    g = Gen(6)
    x, y = g(9, 1920, dtype=torch.bfloat16), g(9, 1920, dtype=torch.bfloat16)
    before = block.Norm("rms", 1e-6, g(1920, dtype=torch.bfloat16))
    r, h = block.residual_norm(x, y, before=before)
    r1, none = block.residual_norm(x, y)
    assert none is None and torch.equal(r1, r)
    x1, h1 = block.residual_norm(r, before=before)
    assert x1 is r
    check_norm([0, 9], 9, r, None, None, h1, dict(before=before))
    x2, y2 = x.clone(), y.clone()
    r2, h2 = block.residual_norm(x2, y2, before=before, out=x2, normed=y2)
    assert r2 is x2 and h2 is y2 and torch.equal(x2, r) and torch.equal(y2, h)
    r3, h3 = block.residual_norm(x[:0], y[:0], before=before)
    assert r3.shape == h3.shape == (0, 1920)


def test_norm_extreme_rows():
    """Rows of one value, zeros, large and small values; rows that are not finite stay alone."""
    cols = 1024
    x = torch.zeros(8, cols, device=DEV)
    x[1] = 5
    x[2], x[2, 0] = 1e15, -1e15
    x[3], x[3, ::2] = 1e-12, -1e-12
    x[4, 7], x[5, 3], x[6, 2] = float("nan"), float("inf"), -float("inf")
    x[7] = torch.linspace(1000, 1000.5, cols)
    good = [0, 1, 2, 3, 7]
    narrow = x[:, ::16].contiguous()
    narrow[4, 7], narrow[5, 3], narrow[6, 2] = float("nan"), float("inf"), -float("inf")
    for kind in ("rms", "layer"):
        # (rows side by side in a wave: neighbours stay apart)
        kw = dict(before=block.Norm(kind, 1e-6))
        _, h = block.residual_norm(narrow, **kw)
        for i in good:
            check_norm([0, 1], 1, narrow[i:i + 1], None, None, h[i:i + 1], kw)
        assert h[4].isnan().all() and not h[5].isfinite().all() and not h[6].isfinite().all()
    for kind in ("rms", "layer"):
        kw = dict(before=block.Norm(kind, 1e-6))
        _, h = block.residual_norm(x, **kw)
        for i in good:
            check_norm([0, 1], 1, x[i:i + 1], None, None, h[i:i + 1], kw)
        assert h[4].isnan().all() and not h[5].isfinite().all() and not h[6].isfinite().all()
    half = x.to(torch.bfloat16)
    r, _ = block.residual_norm(half, torch.zeros_like(half))
    assert torch.equal(r.isnan(), half.isnan()) and torch.equal(r[5], half[5])


# ------------------------------------------------------------------ tables of angles

@pytest.mark.parametrize("axis_dims,scaling,kw", [
    ([8], "none", {}), ([128], "linear", dict(factor=8.0)), ([64], "base", dict(factor=4.0)),
    ([128], "parts", dict(factor=16.0, trained=4096, slow=1.0, fast=32.0, amplitude=1.277)),
    ([16, 24, 24], "none", dict(base=256.0)), ([32, 48, 48], "parts", dict(factor=2.0, trained=64)),
    ([2, 6], "linear", dict(factor=0.5)), ([64, 64, 64, 64], "base", dict(factor=3.0))])
@pytest.mark.parametrize("given", [False, True])
def test_rotation_table(axis_dims, scaling, kw, given):
    rows, axes = 1003, len(axis_dims)
    positions = None
    if axes > 1 or given:
        positions = np.random.default_rng(1).integers(-5, 1 << 20, (rows, axes))
        positions[0], positions[1] = 0, (1 << 31) - 1
    rot = block.rotation_table(sum(axis_dims), rows=None if given else rows, axis_dims=axis_dims,
                               positions=None if positions is None else ints(positions),
                               scaling=scaling, interleaved=True, device=DEV, **kw)
    if positions is None:
        positions = np.arange(rows)[:, None]
    cos, sin, angle = model.rotation_table(axis_dims, positions, scaling=scaling, **kw)
    assert rot.interleaved and rot.positions is None
    # speeds from two 64-bit powers a few steps apart, products and sums of them: 2^-49 of the angle
    far = kw.get("amplitude", 1.0) * 2.0 ** -49 * np.abs(angle)
    close(rot.cos, cos, far + 2.0 ** -50)
    close(rot.sin, sin, far + 2.0 ** -50)


# ------------------------------------------------------------------ rotation

def table(rows, rot):
    freq = 100.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return a.cos().float().to(DEV), a.sin().float().to(DEV)


@pytest.mark.parametrize("dim,rot", [(32, 32), (64, 64), (64, 8), (128, 128), (128, 72), (256, 256),
                                     (256, 16)])
@pytest.mark.parametrize("real", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_rotate(dim, rot, real, pairs, normed):
    """Queries, shared keys and a third tensor of one projection, ragged rows with gaps."""
    g = Gen(dim + rot)
    heads, offsets, starts, tokens = [5, 2, 9], [1, 4, 4, 17], [0, 3, 38], 19
    rows = g(tokens, sum(heads) + 3, dim, dtype=REAL[real])
    xs = list(rows.split(heads + [3], 1)[:3])
    weights = None
    if normed:
        weights = [g(dim, dtype=REAL[real]), None, g(dim)]
    turn = kv8.Rotation(*table(50, rot), interleaved=pairs)
    outs = [torch.full((tokens, h, dim), 7.0, dtype=REAL[real], device=DEV) for h in heads]
    got = block.rotate(xs, turn, ints(offsets), ints(starts), weights=weights, eps=1e-5, outs=outs)
    place = np.zeros(tokens, int)
    inside = np.zeros(tokens, bool)
    for a, e, s in zip(offsets, offsets[1:], starts):
        place[a:e], inside[a:e] = np.arange(s, s + e - a), True
    place = np.minimum(place, 49)
    for i, (x, y) in enumerate(zip(xs, got)):
        want, off = model.rotate(to64(x), to64(turn.cos)[place], to64(turn.sin)[place], pairs, normed,
                                 float(np.float32(1e-5)), to64(weights[i]) if normed else None)
        keep = torch.tensor(inside, device=DEV)
        close(y[keep], want[inside], off[inside])
        assert (y[~keep] == 7).all()


@pytest.mark.parametrize("heads", [1, 7, 8, 16, 17, 33, 1024])
def test_rotate_head_counts_and_in_place(heads):
    """One wave a token and many, tensors ending inside a wave, in place; positions by token, some
    outside of the table."""
    g = Gen(heads)
    tokens, dim = 5, 64
    q, k = g(tokens, heads, dim, dtype=torch.float16), g(tokens, 3, dim, dtype=torch.float16)
    positions = ints([0, 9, -4, 1 << 30, 3])
    turn = kv8.Rotation(*table(10, dim), interleaved=True, positions=positions)
    a, b = block.rotate([q, k], turn)
    at = np.clip(positions.cpu().numpy(), 0, 9)
    for x, y in ((q, a), (k, b)):
        want, off = model.rotate(to64(x), to64(turn.cos)[at], to64(turn.sin)[at], True)
        close(y, want, off)
    q2, k2 = q.clone(), k.clone()
    block.rotate([q2, k2], turn, outs=[q2, k2])
    assert torch.equal(q2, a) and torch.equal(k2, b)
    q3, k3 = q.clone(), k.clone()
    got = block.rotate([q3, k3], turn, outs=[q3, None])
    assert got[0] is q3 and torch.equal(q3, a) and torch.equal(got[1], b) and torch.equal(k3, k)


def test_rotate_norm_alone_and_no_rows():
    g = Gen(1)
    x = g(6, 3, 128, dtype=torch.bfloat16)
    (y,) = block.rotate([x], None, normed=True, eps=0.0)
    want, off = model.rotate(to64(x), None, None, False, True, 0.0)
    close(y, want, off)
    turn = kv8.Rotation(*table(4, 128))
    assert block.rotate([x[:0]], turn)[0].shape == (0, 3, 128)


def test_rotated_keys_are_the_caches():
    """Keys turned here and appended as they are, against keys that append turns: equal to one rounding
    of the rotated key to fp32 and one code."""
    g = Gen(2)
    x = g(70, 2, 64)
    for pairs in (False, True):
        turn = block.rotation_table(64, rows=100, interleaved=pairs, device=DEV)
        args = (ints([[0, 1]]), ints([30]), ints([0, 70]), 70)
        got = []
        for k, rot in ((x, turn), (block.rotate([x], turn, ints([0, 70]), ints([30]))[0], None)):
            cache = kv8.Cache(2, 2, 64, 64, "int8", device=DEV)
            cache.append(k, x, *args, rotation=rot)
            got.append(cache)
        assert (got[0].k.int() - got[1].k.int()).abs().max() <= 1
        assert torch.allclose(got[0].k_scale, got[1].k_scale, rtol=4 * model.U, atol=0)


# ------------------------------------------------------------------ streams and graphs

def test_streams_and_graphs():
    """Another stream than the current one; captured and replayed on new values."""
    g = Gen(9)
    x, y = g(33, 1920, dtype=torch.bfloat16), g(33, 1920, dtype=torch.bfloat16)
    q = g(33, 4, 64, dtype=torch.bfloat16)
    before = block.Norm("layer", 1e-6)
    offsets, starts = ints([0, 20, 33]), ints([5, 0])

    def step(stream=None):
        turn = block.rotation_table(64, rows=64, device=DEV, stream=stream)
        return (*block.residual_norm(x, y, before=before, stream=stream),
                *block.rotate([q], turn, offsets, starts, stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(3):
        x.copy_(g(33, 1920, dtype=torch.bfloat16))
        q.copy_(g(33, 4, 64, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, step())), i


def far_rows(rows, width, dtype, step=1 << 28):
    """Rows so far apart that their elements pass 2^32."""
    return torch.empty((rows - 1) * step + width, dtype=dtype, device=DEV).as_strided((rows, width),
                                                                                      (step, 1))


def test_rows_past_four_gigabytes():
    g = Gen(30)
    near, y = g(18, 256, dtype=torch.bfloat16), g(18, 256, dtype=torch.bfloat16)
    x, h = far_rows(18, 256, torch.bfloat16), far_rows(18, 256, torch.bfloat16)
    x.copy_(near)
    before = block.Norm("rms", 1e-6)
    want = block.residual_norm(near, y, before=before)
    r, n = block.residual_norm(x, y, before=before, out=x, normed=h)
    assert torch.equal(r, want[0]) and torch.equal(n, want[1])
    x.copy_(near)
    turn = kv8.Rotation(*table(20, 64))
    (want,) = block.rotate([near.view(18, 4, 64)], turn)
    (got,) = block.rotate([x.unflatten(1, (4, 64))], turn, outs=[h.unflatten(1, (4, 64))])
    assert torch.equal(got, want)


def test_refusals_of_the_binding():
    g = Gen(40)
    x, y = g(6, 64, dtype=torch.bfloat16), g(6, 64, dtype=torch.bfloat16)
    norm = block.Norm("rms", 1e-6)
    bad_norm = [dict(y=y.half()), dict(y=y[:, :32]), dict(y=y[:5]), dict(y=y.t().contiguous().t()),
                dict(y=y.cpu()), dict(out=x.float()), dict(out=x[:5]), dict(normed=y.float()),
                dict(offsets=ints([0, 6]).long()), dict(offsets=ints([0, 6]).cpu()),
                dict(gate=y[:4]), dict(gate=y[0].half()), dict(gate=y[0, :32]),
                dict(scale=y[:2].t().contiguous().t()), dict(before=block.Norm("batch")),
                dict(before=block.Norm("rms", 1e-6, y[0].half())),
                dict(before=block.Norm("rms", 1e-6, y[0, :32])),
                dict(before=block.Norm("layer", 1e-6, y[0], y[0].float())),
                dict(before=block.Norm("rms", 1e-6, None, y[0])), dict(gate_scale=float("nan")),
                dict(dtype=torch.float64)]
    for kw in bad_norm:
        with pytest.raises((ValueError, TypeError, cfz.CfzError)):
            block.residual_norm(x, **{"y": y, "before": norm, **kw})
    for args in ((x.double(),), (x[0],), (x.cpu(),), (x,)):
        with pytest.raises((ValueError, TypeError, cfz.CfzError)):
            block.residual_norm(*args)
    for kw in (dict(rows=None), dict(rows=-1), dict(positions=ints([1, 2]).long()),
               dict(positions=ints([[1, 2]])), dict(rows=3, positions=ints([1, 2])),
               dict(axis_dims=[4, 4]), dict(axis_dims=[8] * 5), dict(scaling="no"),
               dict(device="cpu"), dict(scaling="parts"), dict(rows=1 << 40)):
        with pytest.raises((ValueError, TypeError, cfz.CfzError)):
            block.rotation_table(64, **{"rows": 4, "device": DEV, **kw})
    q, turn = g(6, 2, 64), block.rotation_table(64, rows=8, device=DEV)
    for args, kw in ((([],), {}), (([q] * 5,), {}), (([q, q.half()],), {}), (([q, q[:5]],), {}),
                     (([q[0]],), {}), (([q.cpu()],), {}), (([q.transpose(1, 2)],), {}),
                     (([q],), dict(offsets=ints([0, 6]).long())), (([q],), dict(starts=ints([0, 1]))),
                     (([q],), dict(weights=[None, None])), (([q],), dict(weights=[q[0, 0].half()])),
                     (([q],), dict(weights=[q[0, 0, :32]])), (([q],), dict(outs=[q.half()])),
                     (([q],), dict(outs=[q[:, :1]])), (([q],), dict(outs=[])),
                     (([q],), dict(normed=False, weights=[q[0, 0]])),
                     (([q],), dict(rotation=None)), (([q[..., :48].contiguous()],), {})):
        with pytest.raises((ValueError, TypeError, cfz.CfzError)):
            block.rotate(*args, **{"rotation": turn, **kw})
