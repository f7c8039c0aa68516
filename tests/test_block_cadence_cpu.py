"""What ``cadence``'s steps refuse about norms and rotations, and when: before a stream is touched and
before a receiver's base, a sum in place or a sender's state moves.  No GPU: as in
``test_kv8_cadence_cpu``."""
import pytest
import torch

from diffusion_activation_residual_amd import block, cadence, cfz, kv8
from test_kv8_cadence_cpu import BATCH, DIM, HEADS, PAGE, QUERIES, TOKENS, Stream, cache, rotation, rows

NQ = BATCH * QUERIES


@pytest.fixture(autouse=True)
def _host_tensors(monkeypatch):
    monkeypatch.setattr(block, "_device", lambda t, what: t.device)


def step(log, monkeypatch, weights=None, heads=2 * HEADS, kv_heads=HEADS, **plan):
    """Two layers of two shares that are there already; weights[1] is the second layer's."""
    for name in ("append", "attend", "select"):
        monkeypatch.setattr(kv8.Cache, name, lambda *a, name=name, **k: log.append(name))
    monkeypatch.setattr(block, "rotate", lambda *a, **k: [log.append("rotate")])
    kw = dict(rotation=rotation(), query_start=3, head_norm=1e-6)
    kw.update(plan)
    plan = cadence.SharePlan(BATCH, TOKENS, QUERIES, PAGE, device="cpu", **kw)
    layers = [[cadence.Share(*(rows(BATCH * n, kv_heads) for _ in "kv")) for n in TOKENS]
              for _ in range(2)]
    q = [rows(NQ, heads) for _ in range(2)]
    cadence.enqueue_layer_attention(plan, layers, [cache(heads=kv_heads) for _ in range(2)], q, q,
                                    [Stream(log), Stream(log)], q_weights=weights)


def ones(n=DIM, skip=0, dtype=torch.bfloat16):
    return torch.ones(n + skip, dtype=dtype)[skip:]


@pytest.mark.parametrize("kw", [
    {}, dict(weights=[None, ones()]), dict(weights=[ones(dtype=torch.float32), ones(skip=8)]),
    dict(query_start=None), dict(head_norm=0.0), dict(head_norm=3e38), dict(head_norm=None),
    dict(kv_heads=16, heads=1024)])
def test_steps_that_fit(kw, monkeypatch):
    log = []
    step(log, monkeypatch, **kw)
    assert log == ["wait"] + ["append", "append", "rotate", "attend"] * 2 + ["wait"]


@pytest.mark.parametrize("kw,why", [
    (dict(weights=[ones(), ones(skip=1)]), "aligned"), (dict(weights=[ones(), ones(skip=4)]), "aligned"),
    (dict(weights=[None, ones(skip=2, dtype=torch.float32)]), "aligned"), (dict(head_norm=1e39), "eps"),
    (dict(kv_heads=17, heads=17 * 61), "heads"),
    (dict(query_start=None, kv_heads=17, heads=17 * 61), "heads"),
    (dict(head_norm=None, kv_heads=17, heads=17 * 61), "heads")])
def test_queries_that_cannot_be_turned_are_refused_before_any_work(kw, why, monkeypatch):
    log = []
    with pytest.raises(cfz.CfzError, match=why):
        step(log, monkeypatch, **kw)
    assert log == []


def test_work_groups_past_the_rotation_limit_are_refused_before_any_work(monkeypatch):
    """65535 items of 40 queries of 1024 heads of 128: 64 waves a token, 2^23 work-groups and more."""
    log = []
    plan = cadence.SharePlan(65535, [32], 40, PAGE, rotation=rotation(64), device="cpu", query_start=0)
    wide = [rows(1, n, 128).expand(65535 * m, -1, -1) for n, m in ((16, 32), (1024, 40))]
    # (no memory for the rows, nor their strides)
    monkeypatch.setattr(kv8, "_rows", lambda t, heads, dim, device, what: heads * dim)
    monkeypatch.setattr(kv8.Cache, "_fits", lambda *a: None)  # (of the other calls)
    c = cache(heads=16, dim=128)
    c.pages = c.desc.pages = plan.pages
    with pytest.raises(cfz.CfzError, match="work-groups"):
        cadence.enqueue_layer_attention(plan, [[cadence.Share(wide[0], wide[0])]], [c], [wide[1]],
                                        [wide[1]], [Stream(log)])
    assert log == []


def features(log, monkeypatch, **second):
    """Two layers; `second` replaces parts of the second one's step."""
    monkeypatch.setattr(block, "residual_norm", lambda *a, **k: log.append("norm"))
    monkeypatch.setattr(cfz, "cfz_compress_group", lambda *a, **k: log.append("compress"))
    monkeypatch.setattr(cfz, "_bf16_ptr", lambda t: t.data_ptr())
    monkeypatch.setattr(cfz, "_ptr", lambda t: t.data_ptr())

    def wide():
        return torch.zeros((4, 64), dtype=torch.bfloat16)

    steps = []
    for change in ({}, second):
        x = wide()
        steps.append(cadence.FeatureStep(**{**dict(x=x, y=wide(), out=x), **change}))
    codes = [torch.zeros(512, dtype=torch.uint8) for _ in steps]
    scales = [torch.zeros(32) for _ in steps]
    cadence.enqueue_layer_features(steps, [10, 20], [wide() for _ in steps], codes, scales, [Stream(log)])


NORM = dict(after=block.Norm("rms"))
GATE = dict(gate=torch.zeros(64, dtype=torch.bfloat16))


@pytest.mark.parametrize("kw", [{}, GATE, NORM, dict(y=None), dict(y=None, before=block.Norm("layer")),
                                dict(y=None, after=block.Norm("none"))])
def test_features_that_fit(kw, monkeypatch):
    log = []
    features(log, monkeypatch, **kw)
    assert log == ["norm", "compress"] * 2


@pytest.mark.parametrize("kw", [GATE, NORM])
def test_a_gate_without_a_block_output_is_refused_before_any_work(kw, monkeypatch):
    """The library's answer to that is the one by which the check knows that only x is left out."""
    log = []
    with pytest.raises((ValueError, cfz.CfzError)):
        features(log, monkeypatch, y=None, **kw)
    assert log == []


def test_a_check_without_any_result():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(cfz.CfzError, match="r and h"):
        block.check_residual_norm(x, None, out=None, normed=None)


@pytest.mark.parametrize("tokens", [0, 4])
def test_a_check_of_neither_norm_nor_rotation(tokens):
    with pytest.raises(cfz.CfzError, match="neither"):
        block.check_rotate([rows(tokens)], None)
    block.check_rotate([rows(tokens)], None, normed=True)


@pytest.mark.parametrize("kw", [{}, dict(rotation=rotation(), query_start=0)])
def test_a_weight_of_queries_that_are_not_normed_is_refused(kw, monkeypatch):
    log = []
    monkeypatch.setattr(kv8.Cache, "attend", lambda *a, **k: log.append("attend"))
    monkeypatch.setattr(block, "rotate", lambda *a, **k: [log.append("rotate")])
    plan = cadence.SharePlan(BATCH, TOKENS, QUERIES, PAGE, device="cpu", **kw)
    with pytest.raises(ValueError, match="head_norm"):
        plan.attend(cache(), rows(NQ, 4), q_weight=ones())
    assert log == []
    plan.attend(cache(), rows(NQ, 4))
    assert log == ["rotate"] * bool(kw) + ["attend"]
