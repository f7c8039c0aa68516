"""Host-side checks of the page management in include/cfz_kv8.h that need no GPU: refusals with the
documented status before any device work (every call below fails validation or is a no-op)."""
import ctypes as C

import pytest

from diffusion_activation_residual_amd import cfz, kv8
from test_kv8_boundary_cpu import A, ODD, cache, ref

lib = cfz._lib


def pages(**kw):
    d = dict(pages=8, batch=2, table_width=4, page_tokens=32, page_table=A, lengths=A, refs=A)
    d.update(kw)
    return kv8.cfz_kv8_pages(**d)


def free(p=pages(), count=1, rows=A, keep=None):
    return lib.cfz_kv8_free(ref(p), count, rows, keep, None)


def fork(p=pages(), count=1, parents=A, children=A):
    return lib.cfz_kv8_fork(ref(p), count, parents, children, None)


def reserve(p=pages(), counts=A, max_new=64, source=A, target=A, missing=A, ws=A, n=1 << 20):
    return lib.cfz_kv8_reserve(ref(p), counts, max_new, source, target, missing, ws, n, None)


def compact(p=pages(), source=A, target=A, live=A, moves=A, ws=A, n=1 << 20):
    return lib.cfz_kv8_compact(ref(p), source, target, live, moves, ws, n, None)


def copy(to=cache(), origin=None, count=1, source=A, target=A, used=None):
    return lib.cfz_kv8_copy(ref(to), ref(origin), count, source, target, used, None)


@pytest.mark.parametrize("call", [free, fork, reserve, compact])
@pytest.mark.parametrize("change,status", [
    (dict(page_tokens=16), cfz.CFZ_ERR_UNSUPPORTED), (dict(pages=-1), cfz.CFZ_ERR_SHAPE),
    (dict(pages=1 << 31), cfz.CFZ_ERR_SHAPE), (dict(batch=0), cfz.CFZ_ERR_SHAPE),
    (dict(batch=65536), cfz.CFZ_ERR_SHAPE), (dict(table_width=0), cfz.CFZ_ERR_SHAPE),
    (dict(table_width=1 << 26), cfz.CFZ_ERR_SHAPE), (dict(page_table=None), cfz.CFZ_ERR_NULL),
    (dict(lengths=None), cfz.CFZ_ERR_NULL), (dict(refs=None), cfz.CFZ_ERR_NULL),
    (dict(refs=A + 2), cfz.CFZ_ERR_ALIGN), (dict(page_table=A + 1), cfz.CFZ_ERR_ALIGN),
])
def test_bad_tables(call, change, status):
    assert call(p=pages(**change)) == status
    assert call(p=None) == cfz.CFZ_ERR_NULL


@pytest.mark.parametrize("call,kw,status", [
    (free, dict(count=-1), cfz.CFZ_ERR_SHAPE), (free, dict(count=65536), cfz.CFZ_ERR_SHAPE),
    (free, dict(rows=None), cfz.CFZ_ERR_NULL), (free, dict(keep=A + 2), cfz.CFZ_ERR_ALIGN),
    (free, dict(p=pages(table_width=1 << 24), count=200), cfz.CFZ_ERR_SHAPE),
    (free, dict(count=0, p=pages(page_table=None)), cfz.CFZ_OK),
    (fork, dict(count=-1), cfz.CFZ_ERR_SHAPE), (fork, dict(parents=None), cfz.CFZ_ERR_NULL),
    (fork, dict(children=None), cfz.CFZ_ERR_NULL), (fork, dict(children=A + 1), cfz.CFZ_ERR_ALIGN),
    (fork, dict(count=0, parents=None, children=None), cfz.CFZ_OK),
    (reserve, dict(counts=None), cfz.CFZ_ERR_NULL), (reserve, dict(max_new=-1), cfz.CFZ_ERR_SHAPE),
    (reserve, dict(max_new=1 << 31), cfz.CFZ_ERR_SHAPE),
    (reserve, dict(p=pages(batch=65535, table_width=1 << 16), max_new=1 << 30), cfz.CFZ_ERR_SHAPE),
    (reserve, dict(source=None), cfz.CFZ_ERR_NULL), (reserve, dict(target=A + 2), cfz.CFZ_ERR_ALIGN),
    (reserve, dict(missing=None), cfz.CFZ_ERR_NULL), (reserve, dict(ws=None), cfz.CFZ_ERR_WORKSPACE),
    (reserve, dict(n=8), cfz.CFZ_ERR_WORKSPACE), (reserve, dict(ws=A + 16), cfz.CFZ_ERR_ALIGN),
    (compact, dict(source=None), cfz.CFZ_ERR_NULL), (compact, dict(live=None), cfz.CFZ_ERR_NULL),
    (compact, dict(moves=A + 2), cfz.CFZ_ERR_ALIGN), (compact, dict(n=8), cfz.CFZ_ERR_WORKSPACE),
    (compact, dict(p=pages(batch=65535, table_width=1 << 20)), cfz.CFZ_ERR_SHAPE),
    (copy, dict(to=None), cfz.CFZ_ERR_NULL), (copy, dict(to=cache(head_dim=96)), cfz.CFZ_ERR_UNSUPPORTED),
    (copy, dict(count=-1), cfz.CFZ_ERR_SHAPE), (copy, dict(count=1 << 31), cfz.CFZ_ERR_SHAPE),
    (copy, dict(source=None), cfz.CFZ_ERR_NULL), (copy, dict(target=A + 2), cfz.CFZ_ERR_ALIGN),
    (copy, dict(used=A + 1), cfz.CFZ_ERR_ALIGN), (copy, dict(to=cache(k=None)), cfz.CFZ_ERR_NULL),
    (copy, dict(to=cache(v=ODD)), cfz.CFZ_ERR_ALIGN),
    (copy, dict(origin=cache(kv_heads=3)), cfz.CFZ_ERR_SHAPE),
    (copy, dict(origin=cache(head_dim=128)), cfz.CFZ_ERR_SHAPE),
    (copy, dict(origin=cache(page_tokens=64)), cfz.CFZ_ERR_SHAPE),
    (copy, dict(origin=cache(format=1)), cfz.CFZ_ERR_SHAPE),
    (copy, dict(origin=cache(k_mean=None)), cfz.CFZ_ERR_NULL),
    (copy, dict(count=0, source=None), cfz.CFZ_OK), (copy, dict(to=cache(pages=0)), cfz.CFZ_OK),
])
def test_refusals(call, kw, status):
    assert call(**kw) == status


def test_workspace_sizes():
    size = lib.cfz_kv8_reserve_workspace_bytes
    # a place a row for a single token; two for more than one (they may start inside a page)
    assert size(C.byref(pages()), 1) == 4 * (2 * 1 + 2 + 2 * 8)
    assert size(C.byref(pages()), 2) == 4 * (2 * 2 + 4 + 2 * 8)
    assert size(C.byref(pages()), 1 << 30) == 4 * (2 * 4 + 8 + 2 * 8)
    assert size(C.byref(pages(page_tokens=5)), 1) == 0
    assert lib.cfz_kv8_compact_workspace_bytes(C.byref(pages(pages=4097))) == 4 * (2 + 4097)
    assert lib.cfz_kv8_compact_workspace_bytes(C.byref(pages(batch=0))) == 0
