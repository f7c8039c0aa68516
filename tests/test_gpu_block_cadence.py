"""The norms, rotations and adapters as the layers of a model use them: queries normed and turned on
their way to the attention over shares, features normed and compressed, and a whole block -- each step
against its model on the values that the step before it left."""
import dataclasses

import numpy as np
import pytest
import torch

from oracle import block as model
from test_gpu_block import Gen, _need_gpu, check_norm, close, ints, to64  # noqa: F401

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_activation_residual_amd import block, cadence, cfz, kv8
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.mark.parametrize("pairs,norm,weighted", [(True, None, False), (False, 1e-6, False),
                                                 (True, 1e-6, True)])
def test_queries_turned_on_the_way(pairs, norm, weighted):
    """Equal to turning them first, eagerly on two streams and in a replayed graph."""
    heads, dim, page, batch, tokens, L = 2, 64, 32, 2, [40, 24], 3
    g = Gen(1)
    turn = block.rotation_table(dim, rows=64, interleaved=pairs, device=DEV)
    plan = cadence.SharePlan(batch, tokens, 24, page, turn, device=DEV, query_start=40, head_norm=norm)
    plain = cadence.SharePlan(batch, tokens, 24, page, turn, device=DEV)
    q = [g(batch * 24, 2 * heads, dim, dtype=BF, size=2) for _ in range(L)]
    weights = [g(dim, dtype=BF), None, g(dim)] if weighted else None
    layers = [[cadence.Share(*(g(batch * n, heads, dim, dtype=BF) for _ in "kv")) for n in tokens]
              for _ in range(L)]

    def run(plan, q, streams, **kw):
        caches = [kv8.Cache(plan.pages, heads, dim, page, device=DEV) for _ in range(L)]
        out = [torch.full_like(t, 5.0) for t in q]
        cadence.enqueue_layer_attention(plan, layers, caches, q, out, streams, **kw)
        return out

    at, starts = ints([0, 24, 48]), ints([40, 40])
    before = [block.rotate([t], turn, at, starts, weights=[weights[l] if weighted else None],
                           normed=norm is not None, eps=norm or 0.0)[0] for l, t in enumerate(q)]
    want = run(plain, before, [torch.cuda.current_stream()])
    kw = dict(q_weights=weights) if weighted else {}
    got = run(plan, q, [torch.cuda.current_stream(), torch.cuda.Stream()], **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    cap = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        kept = run(plan, q, [cap], **kw)
    for i in range(3):
        for t in q:
            t.copy_(g(batch * 24, 2 * heads, dim, dtype=BF))
        graph.replay()
        torch.cuda.synchronize()
        got = run(plan, q, [torch.cuda.current_stream()], **kw)
        assert all(torch.equal(a, b) for a, b in zip(kept, got)), i


def test_plans_that_turn_and_do_not_fit():
    turn = block.rotation_table(64, rows=8, device=DEV)
    args = (1, [4], 4, 32)
    placed = dataclasses.replace(turn, positions=ints([0, 1, 2, 3]))
    for kw in (dict(query_start=0), dict(rotation=placed, query_start=0),
               dict(rotation=turn, query_start=-1), dict(head_norm=-1.0),
               dict(head_norm=float("nan"))):
        with pytest.raises(ValueError):
            cadence.SharePlan(*args, device=DEV, **kw)
    plan = cadence.SharePlan(*args, turn, device=DEV, query_start=0)
    x = torch.zeros(4, 1, 64, dtype=BF, device=DEV)
    cache = kv8.Cache(1, 1, 64, 32, device=DEV)
    streams = [torch.cuda.current_stream()]
    for weights in ([x[0, 0]], []):
        with pytest.raises(ValueError):
            cadence.enqueue_layer_attention(plan, [[cadence.Share(x, x)]], [cache], [x], [x.clone()],
                                            streams, q_weights=weights)
    plan = cadence.SharePlan(*args, turn, device=DEV, query_start=0, head_norm=1e-6)
    for weight in (x[0, 0, :32], x[0, 0].cpu(), x[0]):
        with pytest.raises(ValueError):
            cadence.enqueue_layer_attention(plan, [[cadence.Share(x, x)]], [cache], [x], [x.clone()],
                                            streams, q_weights=[weight])
    assert not cache.k_scale.any()


class Features:
    """Three layers: stream, block outputs, modulation, a sender each."""

    def __init__(self, batch, rows, cols, stream):
        self.g = g = Gen(cols)
        n = batch * rows
        self.x0 = [g(n, cols, dtype=BF) for _ in range(3)]
        self.senders = [cfz.Sender(n, cols, x0=t) for t in self.x0]
        self.x = [g(n, cols, dtype=stream) for _ in range(3)]
        self.y = [g(n, cols, dtype=BF) for _ in range(3)]
        mods = [g(batch, 3 * cols, dtype=BF, size=0.3).chunk(3, 1) for _ in range(3)]
        self.mods = [dict(zip(("gate", "scale", "shift"), m)) for m in mods]
        self.h = [torch.full((n, cols), 7.0, dtype=BF, device=DEV) for _ in range(3)]

    def steps(self):
        return [cadence.FeatureStep(x, y, out=x, before=block.Norm("layer", 1e-6), **m)
                for x, y, m in zip(self.x, self.y, self.mods)]

    def run(self, streams, **change):
        args = dict(steps=self.steps(), senders=[s.handle for s in self.senders], features=self.h,
                    codes=[s.codes for s in self.senders], scales=[s.scales for s in self.senders])
        args.update(change)
        cadence.enqueue_layer_features(**args, streams=streams)

    def tensors(self):
        return [t for s in self.senders for t in (s.codes, s.scales, s.prev, s.err)] + self.x + self.h


@pytest.mark.parametrize("stream", [BF, torch.float32])
def test_features_normed_and_compressed(stream):
    """Equal to the two calls by themselves; on two streams, on one, and in a replayed graph."""
    sides = [Features(2, 21, 192, stream) for _ in range(4)]
    streams = [torch.cuda.current_stream(), torch.cuda.Stream()]
    cap, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    for step in range(4):
        a, b, c, d = sides
        a.run(streams)
        b.run(streams[:1])
        for x, y, m, h, s in zip(c.x, c.y, c.mods, c.h, c.senders):
            block.residual_norm(x, y, before=block.Norm("layer", 1e-6), out=x, normed=h, **m)
            s.compress(h)
        if step == 0:
            d.run(streams[:1])
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=cap):
                d.run([cap, streams[1]])
        else:
            graph.replay()
        torch.cuda.synchronize()
        for other in (b, c, d):
            assert all(torch.equal(p, q) for p, q in zip(a.tensors(), other.tensors())), step
        for side in sides:
            for y in side.y:
                y.mul_(0.5)


def test_features_that_do_not_fit_change_nothing():
    f = Features(1, 8, 64, BF)
    other = Features(1, 8, 128, BF)
    before = [t.clone() for t in f.tensors()]
    streams = [torch.cuda.current_stream()]
    steps, h = f.steps(), f.h

    def last(**kw):
        return steps[:2] + [dataclasses.replace(steps[2], **kw)]

    flat = torch.zeros(9 * 64 + 4, dtype=BF, device=DEV)
    bad = [dict(steps=steps[:2]), dict(steps=last(y=f.y[2][:, :32])), dict(steps=last(y=f.y[2].half())),
           dict(steps=last(out=None)), dict(steps=last(x=f.x[2].cpu())),
           dict(steps=last(before=block.Norm("none", 1e-6, f.y[2][0]))),
           dict(steps=last(before=block.Norm("rms", -1.0))),
           dict(steps=last(gate=f.y[2][:3])), dict(steps=last(offsets=ints([0, 4]).long())),
           dict(steps=last(gate_scale=float("inf"))),
           dict(steps=last(y=flat[4:4 + 8 * 64].view(8, 64))),
           dict(steps=last(x=flat[4:4 + 8 * 64].view(8, 64))),
           dict(features=h[:2] + [h[2][:, :32]]), dict(features=h[:2] + [h[2].float()]),
           dict(features=h[:2] + [None]), dict(senders=[s.handle for s in f.senders[:2]] * 2),
           dict(senders=[s.handle for s in f.senders[:2]] + [f.senders[0].handle]),
           dict(senders=[s.handle for s in f.senders[:2]] + [other.senders[0].handle]),
           dict(codes=[s.codes for s in f.senders[:2]] + [f.senders[2].codes[:16]]),
           dict(scales=[s.scales for s in f.senders[:2]] + [f.senders[2].scales.half()])]
    receiver = cfz.Receiver(8, 64, x0=f.x0[0])
    bad.append(dict(senders=[s.handle for s in f.senders[:2]] + [receiver.handle]))
    for kw in bad:
        with pytest.raises((ValueError, TypeError, cfz.CfzError)):
            f.run(streams, **kw)
    with pytest.raises(ValueError):
        f.run([])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(before, f.tensors()))
    f.run(streams)


def test_a_block_step_by_step():
    """Two sequences (a prompt of 45 tokens, one of 20) and then one token each through a block: norm, the
    shared projection and its adapters, rotation, pages, append, attention, the output's gate and sum.
    Each step against its model on the values that the step before it left.

    Attention: fp16 weights 2^-11, scores of at most 2^8 off by 72 2^-24 reach + 2^-13 in either sum, the
    result's rounding: within 2^-9 sum w|v| + 2^-8 |out| for reach = max sum |q k| scale below 128."""
    g = Gen(20)
    cols, heads, kv, dim, page = 256, 4, 2, 64, 32
    width = (heads + 2 * kv) * dim
    shares = [heads * dim, kv * dim, kv * dim]
    proj, back = g(width, cols, dtype=BF, size=cols ** -0.5), g(cols, heads * dim, dtype=BF, size=0.06)
    a = g(2, 3 * 16, cols, dtype=BF, size=cols ** -0.5)
    adapters = block.Adapters(a, g(2, width, 16, dtype=BF, size=0.25), g(2), slices=shares)
    weights = [g(dim, dtype=BF, size=0.2, mean=1), g(dim, dtype=BF, size=0.2, mean=1)]
    turn = block.rotation_table(32, rows=128, scaling="linear", factor=2.0, interleaved=False,
                                device=DEV)
    mods = dict(zip(("shift", "scale", "gate"), g(2, 3 * cols, dtype=BF, size=0.3).chunk(3, 1)))
    before = block.Norm("rms", 1e-6, g(cols, dtype=BF))
    cache = kv8.Cache(8, kv, dim, page, device=DEV)
    pages = kv8.Pages.empty(8, 2, 4, page, DEV)
    ids = [1, 0]
    for counts in ([45, 20], [1, 1], [1, 1]):
        n = sum(counts)
        at = [0, counts[0], n]
        offsets = ints(at)
        x = g(n, cols, dtype=torch.float32)
        held = pages.lengths.tolist()

        kw = dict(before=before, scale=mods["scale"], shift=mods["shift"])
        _, h = block.residual_norm(x, offsets=offsets, dtype=BF, **kw)
        check_norm(at, n, x, None, None, h, kw)

        base = h @ proj.t()
        qkv = adapters.add(h, base, ints(ids), offsets, max(counts))
        for b in range(2):
            rows = slice(at[b], at[b + 1])
            want, off = model.adapters_add(to64(h[rows]), to64(base[rows]), to64(a[ids[b]]),
                                           to64(adapters.b[ids[b]]), float(adapters.scale[ids[b]]),
                                           shares, "bf16")
            close(qkv[rows], want, off)
        q, k, v = (t.view(n, -1, dim) for t in qkv.split(shares, 1))
        rq, rk = block.rotate([q, k], turn, offsets, pages.lengths, weights=weights)
        place = np.concatenate([np.arange(s, s + c) for s, c in zip(held, counts)])
        for t, y, w in ((q, rq, weights[0]), (k, rk, weights[1])):
            want, off = model.rotate(to64(t), to64(turn.cos)[place], to64(turn.sin)[place], False,
                                     True, float(np.float32(1e-6)), to64(w))
            close(y, want, off)

        moves, missing = pages.reserve(ints(counts), max(counts))
        cache.copy(moves)
        cache.append(rk, v, pages.table, pages.lengths, offsets, max(counts))
        pages.lengths += ints(counts)
        assert int(missing) == 0 and pages.lengths.tolist() == [s + c for s, c in zip(held, counts)]
        out, _ = cache.attend(rq, pages.table, pages.lengths, offsets, max(counts), 4 * page,
                              causal=True)
        for b in range(2):
            length, rows = held[b] + counts[b], slice(at[b], at[b + 1])
            gk, gv = (to64(t) for t in cache.gather(
                pages.table[b:b + 1], ints([0]), ints([0, length]), length, length, torch.float32))
            queries = to64(rq[rows])
            for head in range(heads):
                s = queries[:, head] @ gk[:, head // 2].T * dim ** -0.5
                reach = np.abs(queries[:, head]) @ np.abs(gk[:, head // 2]).T * dim ** -0.5
                assert reach.max() < 128
                s[np.arange(length) > np.arange(held[b], length)[:, None]] = -np.inf
                w = np.exp(s - s.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                want, size = w @ gv[:, head // 2], w @ np.abs(gv[:, head // 2])
                err = np.abs(to64(out[rows, head]) - want)
                assert (err <= 2.0 ** -9 * size + 2.0 ** -8 * np.abs(want)).all()

        y = out.view(n, -1) @ back.t()
        kw = dict(gate=mods["gate"], after=block.Norm("rms", 1e-6), gate_scale=0.5)
        r, none = block.residual_norm(x, y, offsets=offsets, out=x.clone(), **kw)
        assert none is None
        check_norm(at, n, x, y, r, None, kw)
