"""Host numbers that do not fit the library's fields: ctypes would cut them to their low bits, and the
library would then see other sizes than the tensors were checked against.  No GPU: caches over host
tensors; what would be launched is recorded instead."""
import pytest
import torch

from diffusion_activation_residual_amd import cadence, kv8
from test_kv8_cadence_cpu import cache, rows

INTS = dict(dtype=torch.int32)


def ints(*x):
    return torch.tensor(x, **INTS)


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(kv8.Cache, "_call", lambda self, call, stream, *a: made.append(call.__name__))
    return made


def arguments():
    return torch.zeros((1, 4), **INTS), ints(100), ints(0, 8)


@pytest.mark.parametrize("change", [
    dict(q_block=2 ** 32 + 1), dict(q_block=2 ** 31), dict(count=2 ** 32 + 2), dict(first=2 ** 32),
    dict(first=-2 ** 32 + 1), dict(last=2 ** 32), dict(max_q=2 ** 64 + 8), dict(max_kv=2 ** 64 + 100)])
def test_select(calls, change):
    c, q = cache(), rows(8, 4)
    kw = dict(max_q=8, max_kv=100, q_block=4, count=2)
    c.select(q, *arguments(), **kw)
    assert calls == ["cfz_kv8_select"]
    with pytest.raises(ValueError, match="bits"):
        kw.update(change)
        lists = torch.zeros((1, -(-kw["max_q"] // kw["q_block"]) % 64, 2, 2), **INTS)
        c.select(q, *arguments(), blocks=lists, **kw)
    assert calls == ["cfz_kv8_select"]


@pytest.mark.parametrize("change", [dict(q_block=2 ** 32 + 1), dict(max_q=2 ** 64 + 4),
                                    dict(max_kv=2 ** 64 + 100)])
def test_attend(calls, change):
    c, q = cache(), rows(8, 4)
    kw = dict(max_q=8, max_kv=100, q_block=8)
    lists = torch.zeros((1, 1, 2, 3), **INTS)
    c.attend(q, *arguments(), blocks=lists, **kw)
    assert calls == ["cfz_kv8_attend"]
    kw.update(change)
    with pytest.raises(ValueError, match="bits"):
        c.attend(q, *arguments(), blocks=None if "max_q" in change else lists, **kw)
    assert calls == ["cfz_kv8_attend"]


def test_append_and_gather(calls):
    c, k = cache(), rows(8)
    with pytest.raises(ValueError, match="bits"):
        c.append(k, k, *arguments(), 2 ** 64 + 8)
    with pytest.raises(ValueError, match="bits"):
        c.gather(*arguments(), 8, 2 ** 64 + 8)
    with pytest.raises(ValueError, match="bits"):
        c.append(k, k, ints(0).expand(1, 1).as_strided((2 ** 32 + 1, 1), (0, 1)), ints(100),
                 ints(0, 8), 8)
    assert calls == []


def test_share_plans():
    kw = dict(batch=1, share_tokens=[8], queries=1, page_tokens=32, device="cpu")
    for bad in (dict(count=2, q_block=2 ** 32 + 1), dict(count=2 ** 32 + 2), dict(count=4097)):
        with pytest.raises(ValueError):
            cadence.SharePlan(**kw, **bad)
    cadence.SharePlan(**kw, count=4096, q_block=2 ** 31 - 1)
