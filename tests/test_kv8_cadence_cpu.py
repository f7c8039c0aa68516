"""What ``cadence.enqueue_layer_attention`` refuses, and when: a step that does not fit is refused
before a stream is touched and before a receiver's base moves.  No GPU: the caches are descriptions over
host tensors, the streams and the library's launches record that they were reached."""
import ctypes as C
import dataclasses

import pytest
import torch

from diffusion_activation_residual_amd import cadence, cfz, kv8

CPU = torch.device("cpu")
HEADS, DIM, PAGE, BATCH, TOKENS, QUERIES = 2, 64, 32, 2, [8, 16], 4


class Stream:
    device = CPU

    def __init__(self, log):
        self.log = log

    def wait_stream(self, other):
        self.log.append("wait")


def cache(pages=8, heads=HEADS, dim=DIM, page=PAGE, pooled=True, device=CPU):
    """A cache over host memory (the class itself takes GPU tensors only)."""
    c = kv8.Cache.__new__(kv8.Cache)
    c.pages, c.kv_heads, c.head_dim, c.page_tokens, c.device = pages, heads, dim, page, device
    n = pages * heads * dim * page
    c.k, c.v = torch.zeros(n, dtype=torch.int8), torch.zeros(n, dtype=torch.int8)
    c.k_scale = c.v_scale = torch.zeros(pages * heads)
    c.k_mean = torch.zeros(pages * heads * dim) if pooled else None
    c.desc = kv8.cfz_kv8_cache(pages, heads, dim, page, 0, c.k.data_ptr(), c.v.data_ptr(),
                               c.k_scale.data_ptr(), c.v_scale.data_ptr(),
                               c.k_mean.data_ptr() if pooled else None)
    c._ref = C.byref(c.desc)
    return c


def rows(n, heads=HEADS, dim=DIM, dtype=torch.bfloat16):
    return torch.zeros((n, heads, dim), dtype=dtype)


def rotation(rot=DIM, positions=None):
    return kv8.Rotation(torch.ones(64, rot // 2), torch.zeros(64, rot // 2), positions=positions)


def step(log, monkeypatch, plan=None, **change):
    """Two layers of an own share and a received one; `change` replaces parts of the second."""
    plan_kw = dict(rotation=rotation(), q_block=2, count=2, first=0, last=1, device="cpu")
    plan_kw.update(plan or {})
    plan = cadence.SharePlan(BATCH, TOKENS, QUERIES, PAGE, **plan_kw)
    monkeypatch.setattr(cfz, "cfz_decompress_group", lambda *a, **k: log.append("decode"))
    monkeypatch.setattr(kv8.Cache, "append", lambda *a, **k: log.append("append"))
    monkeypatch.setattr(kv8.Cache, "select", lambda *a, **k: log.append("select"))
    monkeypatch.setattr(kv8.Cache, "attend", lambda *a, **k: log.append("attend"))
    monkeypatch.setattr(cfz, "_ptr", lambda t: t.data_ptr())  # (host tensors)

    def layer(name):
        own = cadence.Share(rows(BATCH * TOKENS[0]), rows(BATCH * TOKENS[0]))
        n = BATCH * TOKENS[1]
        got = cadence.Share(rows(n, dtype=torch.float32), rows(n, dtype=torch.float32),
                            receivers=(name, name + 1),
                            codes=(torch.zeros(64, dtype=torch.uint8),) * 2,
                            scales=(torch.zeros(16),) * 2)
        return dict(own=own, got=got, cache=cache(), q=rows(BATCH * QUERIES, 2 * HEADS),
                    out=rows(BATCH * QUERIES, 2 * HEADS))

    parts = [layer(10), layer(20)]
    for key, value in change.items():
        if isinstance(value, dict):
            parts[1][key] = dataclasses.replace(parts[1][key], **value)
        else:
            parts[1][key] = value
    streams = change.get("streams", [Stream(log), Stream(log)])
    cadence.enqueue_layer_attention(plan, [[p["own"], p["got"]] for p in parts],
                                    [p["cache"] for p in parts], [p["q"] for p in parts],
                                    [p["out"] for p in parts], streams)


def test_a_step_that_fits_goes_through(monkeypatch):
    log = []
    step(log, monkeypatch)
    layer = ["decode", "append", "append", "select", "attend"]
    assert log == ["wait"] + layer * 2 + ["wait"]


N0, N1, NQ = BATCH * TOKENS[0], BATCH * TOKENS[1], BATCH * QUERIES
BAD = {
    "v rows": dict(own=dict(v=rows(N0 - 1))),
    "v rows of a received share": dict(got=dict(v=rows(N1 + 1, dtype=torch.float32))),
    "k heads": dict(own=dict(k=rows(N0, HEADS + 1))),
    "v heads": dict(own=dict(v=rows(N0, HEADS + 1))),
    "k dim": dict(own=dict(k=rows(N0, dim=128))),
    "k and v types": dict(own=dict(v=rows(N0, dtype=torch.float32))),
    "k type": dict(own=dict(k=rows(N0, dtype=torch.float64), v=rows(N0, dtype=torch.float64))),
    "k heads apart": dict(own=dict(k=rows(N0, 2 * HEADS)[:, ::2])),
    "k rows overlap": dict(own=dict(k=rows(1).expand(N0, -1, -1))),
    "k stride": dict(own=dict(k=torch.zeros((N0, HEADS * DIM + 4), dtype=torch.bfloat16)
                              [:, :HEADS * DIM].unflatten(1, (HEADS, DIM)))),
    "k alignment": dict(own=dict(k=torch.zeros(N0 * HEADS * DIM + 4, dtype=torch.bfloat16)[4:]
                                 .view(N0, HEADS, DIM))),
    "q heads": dict(q=rows(NQ, 3), out=rows(NQ, 3)),
    "q dim": dict(q=rows(NQ, 4, 128), out=rows(NQ, 4, 128)),
    "q type": dict(q=rows(NQ, 4, dtype=torch.float32), out=rows(NQ, 4, dtype=torch.float32)),
    "too many query heads": dict(q=rows(NQ, 65 * HEADS), out=rows(NQ, 65 * HEADS)),
    "out rows": dict(out=rows(NQ + 1, 4)),
    "out heads": dict(out=rows(NQ, 2)),
    "out type": dict(out=rows(NQ, 4, dtype=torch.float16)),
    "out rows overlap": dict(out=rows(1, 4).expand(NQ, -1, -1)),
    "no mean keys": dict(cache=cache(pooled=False)),
    "cache device": dict(cache=cache(device=torch.device("cuda:1"))),
    "cache dim": dict(cache=cache(dim=96), own=dict(k=rows(N0, dim=96), v=rows(N0, dim=96)),
                      got=dict(k=rows(N1, dim=96), v=rows(N1, dim=96)), q=rows(NQ, 4, 96),
                      out=rows(NQ, 4, 96)),
    "one scale tensor": dict(got=dict(scales=(torch.zeros(16),))),
    "codes alignment": dict(got=dict(codes=(torch.zeros(64, dtype=torch.uint8),
                                            torch.zeros(72, dtype=torch.uint8)[8:]))),
    "closed receiver": dict(got=dict(receivers=(20, None))),
    "one receiver twice": dict(got=dict(receivers=(20, 20))),
    "no streams": dict(streams=[]),
}
BAD_PLANS = {
    "rotation of 12": dict(rotation=rotation(12)),
    "rotation past the head": dict(rotation=rotation(128)),
    "rotation type": dict(rotation=kv8.Rotation(torch.ones(64, 32).double(),
                                                torch.ones(64, 32).double())),
    "positions": dict(rotation=rotation(positions=torch.zeros(N0, dtype=torch.int32))),
    "scale 0": dict(scale=0.0),
    "scale NaN": dict(scale=float("nan")),
    "scale under fp32": dict(scale=1e-60),
    "long lists": dict(count=5000),
}


@pytest.mark.parametrize("what", BAD)
def test_a_layer_that_does_not_fit_is_refused_before_any_work(what, monkeypatch):
    log = []
    with pytest.raises((ValueError, TypeError, cfz.CfzError)):
        step(log, monkeypatch, **BAD[what])
    assert log == []


@pytest.mark.parametrize("what", BAD_PLANS)
def test_a_plan_that_does_not_fit_is_refused_before_any_work(what, monkeypatch):
    log = []
    with pytest.raises((ValueError, TypeError, cfz.CfzError)):
        step(log, monkeypatch, plan=BAD_PLANS[what])
    assert log == []


def test_work_groups_past_the_limit_are_refused_before_any_work(monkeypatch):
    log = []
    plan = cadence.SharePlan(1 << 13, [32], 1, PAGE, device="cpu")
    wide = [rows(1, 512).expand(n, -1, -1) for n in (32 << 13, 1 << 13)]  # (no memory for the rows)
    monkeypatch.setattr(cfz, "cfz_decompress_group", lambda *a, **k: log.append("decode"))
    monkeypatch.setattr(cadence, "_whole_rows", lambda *a: None)          # ... nor their strides checked
    c = cache(heads=512)
    c.pages = c.desc.pages = plan.pages
    with pytest.raises(cfz.CfzError, match="work-groups"):
        cadence.enqueue_layer_attention(plan, [[cadence.Share(wide[0], wide[0])]], [c], [wide[1]],
                                        [wide[1]], [Stream(log)])
    assert log == []


def test_a_sender_among_the_receivers_is_refused_before_any_work(monkeypatch):
    log = []
    desc = {role: cfz.make_desc(16, 64, role=role) for role in (cfz.CFZ_SENDER, cfz.CFZ_RECEIVER)}
    monkeypatch.setattr(cfz, "_sizes", {})
    monkeypatch.setattr(cfz, "_codecs", {})
    cfz._record(20, desc[cfz.CFZ_RECEIVER])
    cfz._record(21, desc[cfz.CFZ_SENDER])
    big = dict(codes=(torch.zeros(512, dtype=torch.uint8),) * 2, scales=(torch.zeros(32),) * 2)
    with pytest.raises(ValueError, match="receiver"):
        step(log, monkeypatch, got=dict(receivers=(20, 21), **big))
    assert log == []
    cfz._record(21, desc[cfz.CFZ_RECEIVER])
    step(log, monkeypatch, got=dict(receivers=(20, 21), **big))
    assert "attend" in log
    with pytest.raises(TypeError, match="scales"):
        step([], monkeypatch, got=dict(receivers=(20, 21), codes=big["codes"],
                                       scales=(torch.zeros(32), torch.zeros(32).double())))
    cfz._record(21, cfz.make_desc(16, 64, bits=2, group=32, role=cfz.CFZ_RECEIVER))
    del log[:]
    with pytest.raises(ValueError, match="codec"):
        step(log, monkeypatch, got=dict(receivers=(20, 21), **big))
    assert log == []


def test_streams_are_joined_when_a_launch_fails(monkeypatch):
    log = []

    def fail(*a, **k):
        raise RuntimeError("out of memory")

    plan = cadence.SharePlan(1, [8], 4, PAGE, device="cpu")
    monkeypatch.setattr(kv8.Cache, "append", fail)
    share = cadence.Share(rows(8), rows(8))
    with pytest.raises(RuntimeError, match="out of memory"):
        cadence.enqueue_layer_attention(plan, [[share]], [cache()], [rows(4, 4)], [rows(4, 4)],
                                        [Stream(log), Stream(log)])
    assert log == ["wait", "wait"]
