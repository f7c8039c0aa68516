"""The page management's binding without a GPU: tables over host tensors; what would be launched is
recorded instead."""
import ctypes as C
import weakref

import pytest
import torch

from diffusion_activation_residual_amd import kv8

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
    assert len(queued) == 1 and len(queued[0]) >= 4
