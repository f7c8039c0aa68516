"""Attention over the 8-bit cache whose pages have value scales of any size beside each other.

The bound is that of tests/test_gpu_kv8.py with the loss of small weights taken row by row: a weight
that fp16 holds as a subnormal number (or not at all) is off by at most 2^-31 of the largest product of
a weight and its page's value scale z, where a page whose codes count as zeros has the z at
which its weights are carried: 2^-32 beside pages with a z from there to 2^32, 2^-100 beside others.
What value scales of 2^-100 or less hold counts as 0: at most 2^-100 qmax."""
import numpy as np
import pytest
import torch

import test_gpu_kv8 as base
from oracle import kv8 as model
from test_gpu_kv8 import DEV, REAL, Both, cumulative, ints, say, to64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_activation_residual_amd import kv8

_need_gpu = base._need_gpu


def exact(x, q, table, length, causal, scale, half):
    """out, lse and their bounds for one sequence."""
    n, heads, dim = q.shape
    group, qmax = heads // x.heads, model.QMAX[x.fmt]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    lse, ltol = np.full((n, heads), -np.inf), np.zeros((n, heads))
    at = np.arange(length)
    for head in range(x.heads):
        k, v, live = x.model.dense(x.table[table], head, 0, length)
        z = np.zeros(length)
        for t in np.flatnonzero(live):
            z[t] = x.model.vs[x.table[table][t // x.page], head]
        for i in range(n):
            see = live & (at <= length - n + i) if causal else live
            if not see.any():
                continue
            zs = z[see]
            near = ((zs > 2.0 ** -32) & (zs <= 2.0 ** 32)).any()
            carried = np.where(zs > 2.0 ** -100, zs, 2.0 ** (-32 if near else -100))
            for h in range(head * group, (head + 1) * group):
                s = scale * (k[see] @ q[i, h])
                w = np.exp(s - s.max())
                out[i, h] = w @ v[see] / w.sum()
                lse[i, h] = s.max() + np.log(w.sum())
                size = w @ np.abs(v[see]) / w.sum()
                e = ((dim + 8) * 2.0 ** -24 * scale * (np.abs(k[see]) @ np.abs(q[i, h])).max() +
                     2.0 ** -21 * 2.0 ** 8)
                lost = length * 2.0 ** -31 * (w * carried).max() / w.sum() + 2.0 ** -100
                tol[i, h] = ((2.0 ** -11 + 2 * e + 2 * length * 2.0 ** -24) * size + lost * qmax)
                ltol[i, h] = e + length * 2.0 ** -24 + 2.0 ** -21 * max(1, abs(lse[i, h]))
    # (results under the smallest normal number of the output type are rounded to its grid)
    return out, lse, tol * (1 + half) + half * np.abs(out) + 2.0 ** -134, ltol


def check(x, counts, group, causal, lengths=None, dtype="bf16", size=1.0, scale=None, max_q=None):
    lengths = x.held if lengths is None else lengths
    q = x.rows(sum(counts), x.heads * group, REAL[dtype], size)
    scale = x.dim ** -0.5 if scale is None else scale
    say(f"[gpu] attend q {[c for c in counts if c]} over {max(lengths)} keys, causal {causal}")
    out, lse = x.cache.attend(q, ints(x.table), ints(lengths), cumulative(counts),
                              max(counts) if max_q is None else max_q, x.table.shape[1] * x.page,
                              causal=causal, scale=scale)
    torch.cuda.synchronize()
    half, at = torch.finfo(REAL[dtype]).eps / 2, 0
    for b, c in enumerate(counts):
        if c == 0:
            continue
        want, wl, tol, ltol = exact(x, to64(q[at:at + c]), b, lengths[b], causal, scale, half)
        got, gl = to64(out[at:at + c]), to64(lse[at:at + c])
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(gl), empty) and not got[empty].any()
        assert np.isfinite(got).all() and np.isfinite(gl[~empty]).all()
        worst = (np.abs(got - want) / tol)[~empty].max(initial=0)
        worst_l = (np.abs(gl[~empty] - wl[~empty]) / ltol[~empty]).max(initial=0)
        say(f"      sequence {b}: {worst:.3f} of the bound, lse {worst_l:.3f}")
        assert worst <= 1 and worst_l <= 1
        at += c


def sized(dim, page, fmt, sizes, seed, short=5):
    """One sequence, its pages' values multiplied by `sizes`; the last page has `short` empty slots."""
    x = Both(1, len(sizes), 1, dim, page, fmt, seed=seed)
    k, v = (x.rows(len(sizes) * page - short, dtype=torch.float32) for _ in range(2))
    for i, s in enumerate(sizes):
        v[page * i:page * (i + 1)] *= s
    x.append([len(k)], k, v)
    x.check()
    return x


PATTERNS = {
    "zeros then large": (0.0, 0.0, 1e10, 0.0),
    "zeros then huge": (0.0, 1.0, 1e30, 0.0),
    "large then zeros": (3e36, 0.0, 0.0, 1.0),
    "rising": (1e-38, 1e-28, 1e-12, 1.0, 1e15, 1e36),
    "falling": (1e36, 1e14, 1.0, 1e-13, 1e-29, 1e-38),
    "tiny and zero": (0.0, 1e-26, 0.0, 1e-25),
    "zero": (0.0, 0.0),
    "inside the ordinary range": (1e-9, 0.0, 1e9, 1.0),
}


@pytest.mark.parametrize("rows", [1, 40, 100, 200, 300])
@pytest.mark.parametrize("pattern", PATTERNS)
def test_attend_value_scales_of_any_size(pattern, rows):
    x = sized(64, 32, "int8", PATTERNS[pattern], seed=40)
    check(x, [rows], 1, False)
    check(x, [rows], 1, True)
    # sharp scores: what a row sees may be one page alone
    check(x, [rows], 1, True, size=8.0)


@pytest.mark.parametrize("rows,dtype", [(1, "f16"), (20, "bf16"), (100, "bf16"), (200, "bf16")])
@pytest.mark.parametrize("pattern", ["zeros then large", "rising", "falling"])
def test_attend_value_scales_of_any_size_at_128(pattern, rows, dtype):
    sizes = PATTERNS[pattern]
    if dtype == "f16":  # what fp16 results hold
        sizes = [min(s, 1e4) for s in sizes]
    x = sized(128, 64, "e4m3", sizes, seed=41)
    check(x, [rows], 2, False, dtype=dtype)
    check(x, [rows], 2, True, dtype=dtype, size=4.0)


@pytest.mark.parametrize("joined", [True, False])
@pytest.mark.parametrize("dim,rows", [(64, 1), (128, 3), (64, 100), (128, 100), (128, 200), (64, 300)])
def test_attend_scales_that_change_far_into_a_sequence(dim, rows, joined):
    """Pages looked up later than the first ones leave the ordinary range, up and down; with many
    sequences (empty ones) a work-group takes a whole tile, else a tile is cut and joined."""
    page, far = 128, 260 if rows > 100 else 70
    sizes = [0.0, 1.0, 1e-28, 1e34]
    x = sized(dim, page, "int8", sizes, seed=42, short=0)  # (each page is used in several places)
    zero, one, tiny, huge = x.table[0]
    row = np.array([zero] * far + [one, tiny] + [one] * far + [huge, zero, zero])
    x.table = np.array([row, [zero] * far + [tiny] * (far + 4) + [zero]])
    x.held = [len(row) * page - 7, len(row) * page]
    others = 0 if joined else 1030
    x.table = np.concatenate([np.repeat(x.table[:1], others, 0), x.table])
    few = min(rows, 4)
    for lengths in (x.held, [(2 * far + 2) * page, (far + 3) * page]):
        check(x, [0] * others + [few, few], 1, False, lengths=[0] * others + list(lengths),
              max_q=rows)


@pytest.mark.parametrize("rows", [1, 100])
def test_attend_many_keys_of_zero_values(rows):
    """2^22 + 2^21 keys whose values are zeros, and flat scores: the sum of the weights stays finite.
    (A lane adds its weights step by step, at most n / 64 of them: below 2^17 roundings of 2^-24.)"""
    page, n = 128, (1 << 22) + (1 << 21)
    cache = kv8.Cache(1, 1, 64, page, "int8", device=DEV)
    zero = torch.zeros((page, 1, 64), dtype=torch.bfloat16, device=DEV)
    cache.append(zero + 1, zero, ints([[0]]), ints([0]), ints([0, page]), page)
    table = torch.zeros((1, n // page), dtype=torch.int32, device=DEV)
    q = torch.zeros((rows, 1, 64), dtype=torch.bfloat16, device=DEV)
    q[rows // 2:] = 1.0  # a score of 64 / 8 for every key
    out, lse = cache.attend(q, table, ints([n]), ints([0, rows]), rows, n)
    want = np.log(n) + np.where(np.arange(rows) < rows // 2, 0.0, 8.0)
    assert not out.any()
    assert np.abs(to64(lse)[:, 0] - want).max() <= 2.0 ** -7 + 2.0 ** -13


@pytest.mark.parametrize("rows", [1, 100, 300])
def test_scales_that_change_between_replays_of_a_graph(rows):
    """Which way the denominators are summed is seen on the device, replay by replay."""
    x = sized(64, 32, "int8", [1.0] * 40, seed=43)
    q, table, held = x.rows(rows), ints(x.table), ints(x.held)
    args = (q, table, held, cumulative([rows]), rows, 40 * 32)
    x.cache.attend(*args)
    torch.cuda.synchronize()
    ordinary = x.cache.v_scale.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = x.cache.attend(*args)
    for far in (None, 1e20, None, 0.0, 1e-20):
        x.cache.v_scale.copy_(ordinary)
        if far is not None:
            x.cache.v_scale[table[0, 7::9].long()] = far
        graph.replay()
        want, wl = x.cache.attend(*args)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl) and torch.isfinite(lse).all()
        # the scores do not depend on the values: two results, each off by 2^-21 2^8 (the exponent with
        # the value scale's logarithm in it) and by the roundings of sum and logarithm
        if far is None:
            base_lse = wl.clone()
        else:
            assert (wl - base_lse).abs().max() <= 2.0 ** -13 * 2 + 2.0 ** -20 * base_lse.abs().max()
