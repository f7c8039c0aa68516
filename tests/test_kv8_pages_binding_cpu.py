"""The page management's binding without a GPU: tables over host tensors; what would be launched is
recorded instead."""
import ctypes as C
import weakref

import pytest
import torch

from diffusion_activation_residual_amd import cfz, kv8
from test_kv8_boundary_cpu import A
from test_kv8_cadence_cpu import cache
from test_kv8_pages_boundary_cpu import pages

CPU = torch.device("cpu")


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def table(pages=8, batch=2, width=4, page=32):
    """A ``Pages`` over host memory (the class itself takes GPU tensors only)."""
    p = kv8.Pages.__new__(kv8.Pages)
    p.device, p.page_tokens = CPU, page
    p.table = torch.full((batch, width), -1, dtype=torch.int32)
    p.lengths, p.refs = torch.zeros(batch, dtype=torch.int32), torch.zeros(pages, dtype=torch.int32)
    p.desc = kv8.cfz_kv8_pages(pages, batch, width, page, p.table.data_ptr(), p.lengths.data_ptr(),
                               p.refs.data_ptr())
    p._ref = C.byref(p.desc)
    return p


@pytest.mark.parametrize("call", [lambda p: p.reserve(ints(1, 1), 1), lambda p: p.compact()])
def test_what_a_call_allocates_is_held_until_it_is_queued(call, monkeypatch):
    """Memory given back before the launch may be another thread's by then."""
    made, queued = [], []

    def empty(device, stream, shape, dtype):
        t = torch.empty(shape, dtype=dtype)
        made.append((t.data_ptr(), weakref.ref(t)))
        return t

    def queue(call, device, stream, *args):
        for at, held in made:
            if at in args:
                assert held() is not None, f"{call.__name__}: {at:#x} is free again"
        queued.append([at for at, _ in made if at in args])

    monkeypatch.setattr(kv8, "_empty_on", empty)
    monkeypatch.setattr(kv8, "_queue", queue)
    call(table())
    assert len(queued) == 1 and len(queued[0]) >= 2


@pytest.mark.parametrize("make,names", [
    (table, ("table", "lengths", "refs")), (cache, ("k", "v", "k_scale", "v_scale", "k_mean")),
    (lambda: cache(pooled=False), ("k", "k_mean"))])
def test_tensors_that_are_known_by_their_address_stay(make, names):
    held = make()
    for name in names:
        t = getattr(held, name)
        for other in (torch.zeros(3) if t is None else t.clone(), None if t is not None else t):
            if other is t:
                continue
            with pytest.raises(ValueError, match=name):
                setattr(held, name, other)
            assert getattr(held, name) is t
        if t is None:
            continue
        at, want = t.data_ptr(), t.clone() + 1
        setattr(held, name, t.add_(1))  # as ``held.name += 1`` does
        assert getattr(held, name).data_ptr() == at and torch.equal(getattr(held, name), want)


def test_lengths_go_on_in_place():
    p = table()
    with pytest.raises(ValueError, match="lengths"):
        p.lengths = p.lengths + ints(3, 4)
    p.lengths += ints(3, 4)
    assert p.lengths.tolist() == [3, 4] and p.desc.lengths == p.lengths.data_ptr()


@pytest.mark.parametrize("change,status", [
    (dict(left_out=None), cfz.CFZ_ERR_NULL), (dict(left_out=A + 2), cfz.CFZ_ERR_ALIGN),
    (dict(counts=None), cfz.CFZ_ERR_NULL), (dict(source=None), cfz.CFZ_ERR_NULL),
    (dict(max_new=-1), cfz.CFZ_ERR_SHAPE), (dict(ws=None), cfz.CFZ_ERR_WORKSPACE)])
def test_refusals_of_reserve_rows(change, status):
    kw = dict(counts=A, max_new=64, source=A, target=A, missing=A, left_out=A, ws=A)
    kw.update(change)
    assert kv8._lib.cfz_kv8_reserve_rows(C.byref(pages()), *kw.values(), 1 << 20, None) == status
