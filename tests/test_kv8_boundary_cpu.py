"""Host-side checks of include/cfz_kv8.h that need no GPU: exported functions, and refusals with
the documented status before any device work (every call below fails validation or is a
no-op)."""
import ctypes as C
import os
import re

import pytest

from diffusion_activation_residual_amd import cfz, kv8

A, ODD = 0x10000, 0x10008  # fake device addresses, never dereferenced
HEADER = os.path.join(os.path.dirname(cfz.HEADER_PATH), "cfz_kv8.h")


def cache(**kw):
    d = dict(pages=8, kv_heads=2, head_dim=64, page_tokens=32, format=0, k=A, v=A, k_scale=A,
             v_scale=A, k_mean=A)
    d.update(kw)
    return kv8.cfz_kv8_cache(**d)


def batch(**kw):
    d = dict(batch=1, table_width=4, page_table=A, offsets=A, lengths=A, tokens=16, max_rows=16)
    d.update(kw)
    return kv8.cfz_kv8_batch(**d)


def rotation(**kw):
    d = dict(cos=A, sin=A, positions=None, table_rows=10, rot_dim=64, interleaved=0)
    d.update(kw)
    return kv8.cfz_kv8_rotation(**d)


def lists(**kw):
    d = dict(blocks=A, count=4, q_block=1)
    d.update(kw)
    return kv8.cfz_kv8_blocks(**d)


def ref(x):
    return None if x is None else C.byref(x)


def append(c=cache(), b=batch(), dtype=0, k=A, v=A, ks=128, vs=128, rot=None):
    return cfz._lib.cfz_kv8_append(ref(c), ref(b), dtype, k, v, ks, vs, ref(rot), None)


def gather(c=cache(), b=batch(), dtype=0, k=A, v=A):
    return cfz._lib.cfz_kv8_gather(ref(c), ref(b), dtype, k, v, None)


def attend(c=cache(), b=batch(), dtype=0, q=A, qs=256, heads=4, scale=1.0, max_kv=128, bl=None,
           out=A, os_=256, lse=A, ws=None, n=0):
    return cfz._lib.cfz_kv8_attend(ref(c), ref(b), dtype, q, qs, heads, 0, scale, max_kv, ref(bl),
                                   out, os_, lse, ws, n, None)


def select(c=cache(), b=batch(), dtype=0, q=A, qs=256, heads=4, max_kv=128, first=0, last=0,
           bl=lists(), ws=A, n=1 << 20):
    return cfz._lib.cfz_kv8_select(ref(c), ref(b), dtype, q, qs, heads, 0, max_kv, first, last,
                                   ref(bl), ws, n, None)


def test_header_functions_are_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(cfz_kv8_[a-z_0-9]+)\s*\(", text))
    assert names == set(kv8._SIGNATURES)
    for name in names:
        assert hasattr(cfz._lib, name)


CALLS = [append, gather, attend, select]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("change,status", [
    (dict(format=2), cfz.CFZ_ERR_UNSUPPORTED),
    (dict(head_dim=96), cfz.CFZ_ERR_UNSUPPORTED),
    (dict(head_dim=0), cfz.CFZ_ERR_UNSUPPORTED),
    (dict(page_tokens=16), cfz.CFZ_ERR_UNSUPPORTED),
    (dict(kv_heads=0), cfz.CFZ_ERR_SHAPE),
    (dict(pages=-1), cfz.CFZ_ERR_SHAPE),
    (dict(pages=1 << 31), cfz.CFZ_ERR_SHAPE),
    (dict(k=None), cfz.CFZ_ERR_NULL),
    (dict(v_scale=None), cfz.CFZ_ERR_NULL),
    (dict(v=ODD), cfz.CFZ_ERR_ALIGN),
    (dict(k_mean=ODD), cfz.CFZ_ERR_ALIGN),
])
def test_bad_caches(call, change, status):
    assert call(c=cache(**change)) == status
    assert cfz.cfz_last_error()


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), cfz.CFZ_ERR_SHAPE),
    (dict(batch=65536), cfz.CFZ_ERR_SHAPE),
    (dict(table_width=0), cfz.CFZ_ERR_SHAPE),
    (dict(table_width=1 << 26), cfz.CFZ_ERR_SHAPE),
    (dict(tokens=-1), cfz.CFZ_ERR_SHAPE),
    (dict(tokens=1 << 31), cfz.CFZ_ERR_SHAPE),
    (dict(max_rows=-1), cfz.CFZ_ERR_SHAPE),
    (dict(page_table=None), cfz.CFZ_ERR_NULL),
    (dict(offsets=None), cfz.CFZ_ERR_NULL),
    (dict(lengths=None), cfz.CFZ_ERR_NULL),
    (dict(lengths=A + 2), cfz.CFZ_ERR_ALIGN),
])
def test_bad_batches(call, change, status):
    assert call(b=batch(**change)) == status


@pytest.mark.parametrize("call", CALLS)
def test_null_structures_and_types(call):
    assert call(c=None) == cfz.CFZ_ERR_NULL
    assert call(b=None) == cfz.CFZ_ERR_NULL
    assert call(dtype=3) == cfz.CFZ_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", CALLS)
def test_nothing_to_do_is_ok(call):
    for change in (dict(batch=0), dict(tokens=0), dict(max_rows=0)):
        assert call(b=batch(page_table=None, offsets=None, lengths=None, **change)) == cfz.CFZ_OK


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), cfz.CFZ_ERR_NULL), (dict(v=None), cfz.CFZ_ERR_NULL),
    (dict(k=ODD), cfz.CFZ_ERR_ALIGN), (dict(ks=127), cfz.CFZ_ERR_SHAPE),
    (dict(ks=120), cfz.CFZ_ERR_SHAPE), (dict(vs=132), cfz.CFZ_ERR_SHAPE),
    (dict(rot=rotation(rot_dim=4)), cfz.CFZ_ERR_SHAPE),
    (dict(rot=rotation(rot_dim=72)), cfz.CFZ_ERR_SHAPE),
    (dict(rot=rotation(rot_dim=12)), cfz.CFZ_ERR_SHAPE),
    (dict(rot=rotation(table_rows=0)), cfz.CFZ_ERR_SHAPE),
    (dict(rot=rotation(cos=None)), cfz.CFZ_ERR_NULL),
    (dict(rot=rotation(sin=ODD)), cfz.CFZ_ERR_ALIGN),
    (dict(rot=rotation(positions=A + 1)), cfz.CFZ_ERR_ALIGN),
])
def test_append_refusals(kw, status):
    assert append(**kw) == status


def test_gather_refusals():
    assert gather(k=ODD) == cfz.CFZ_ERR_ALIGN
    assert gather(k=None, v=None) == cfz.CFZ_OK


QUERY_REFUSALS = [
    (dict(q=None), cfz.CFZ_ERR_NULL), (dict(q=ODD), cfz.CFZ_ERR_ALIGN),
    (dict(dtype=2), cfz.CFZ_ERR_UNSUPPORTED), (dict(heads=3), cfz.CFZ_ERR_SHAPE),
    (dict(heads=0), cfz.CFZ_ERR_SHAPE), (dict(heads=130, qs=130 * 64), cfz.CFZ_ERR_SHAPE),
    (dict(qs=255), cfz.CFZ_ERR_SHAPE), (dict(qs=260), cfz.CFZ_ERR_SHAPE),
    (dict(max_kv=-1), cfz.CFZ_ERR_SHAPE), (dict(max_kv=129), cfz.CFZ_ERR_SHAPE),
    (dict(bl=lists(count=0)), cfz.CFZ_ERR_SHAPE), (dict(bl=lists(count=4097)), cfz.CFZ_ERR_SHAPE),
    (dict(bl=lists(q_block=0)), cfz.CFZ_ERR_SHAPE), (dict(bl=lists(blocks=None)), cfz.CFZ_ERR_NULL),
    (dict(bl=lists(blocks=A + 2)), cfz.CFZ_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", QUERY_REFUSALS + [
    (dict(out=None), cfz.CFZ_ERR_NULL), (dict(out=ODD), cfz.CFZ_ERR_ALIGN),
    (dict(os_=192), cfz.CFZ_ERR_SHAPE), (dict(scale=0.0), cfz.CFZ_ERR_SHAPE),
    (dict(scale=-1.0), cfz.CFZ_ERR_SHAPE), (dict(scale=float("nan")), cfz.CFZ_ERR_SHAPE),
    (dict(scale=float("inf")), cfz.CFZ_ERR_SHAPE),
])
def test_attend_refusals(kw, status):
    assert attend(**kw) == status


@pytest.mark.parametrize("kw,status", QUERY_REFUSALS + [
    (dict(bl=None), cfz.CFZ_ERR_NULL), (dict(c=cache(k_mean=None)), cfz.CFZ_ERR_NULL),
    (dict(first=-1), cfz.CFZ_ERR_SHAPE), (dict(first=3, last=2), cfz.CFZ_ERR_SHAPE),
    (dict(ws=None), cfz.CFZ_ERR_WORKSPACE), (dict(n=16), cfz.CFZ_ERR_WORKSPACE),
    (dict(ws=A + 16), cfz.CFZ_ERR_ALIGN),
])
def test_select_refusals(kw, status):
    assert select(**kw) == status


def test_attend_workspace_is_checked():
    c, b = cache(page_tokens=128, kv_heads=1), batch(table_width=512, tokens=1, max_rows=1)
    need = cfz._lib.cfz_kv8_attend_workspace_bytes(C.byref(c), C.byref(b), 1, 65536, None)
    assert need > 0  # a long cache and one row: the keys are split
    kw = dict(c=c, b=b, qs=64, os_=64, heads=1, max_kv=65536)
    assert attend(**kw) == cfz.CFZ_ERR_WORKSPACE
    assert attend(ws=A, n=need - 1, **kw) == cfz.CFZ_ERR_WORKSPACE
    assert attend(ws=A + 16, n=need, **kw) == cfz.CFZ_ERR_ALIGN
    short = cfz._lib.cfz_kv8_attend_workspace_bytes(C.byref(c), C.byref(b), 1, 64, None)
    assert short == 0
    assert cfz._lib.cfz_kv8_attend_workspace_bytes(C.byref(c), C.byref(b), 0, 64, None) == 0


def test_launches_past_the_grid_limit_are_refused():
    b = batch(batch=65535, tokens=(1 << 31) - 1, max_rows=(1 << 31) - 1)
    for call in CALLS:
        assert call(b=b) in (cfz.CFZ_ERR_SHAPE, cfz.CFZ_ERR_WORKSPACE)


def test_row_and_grid_limits():
    b = batch(batch=1, tokens=1 << 25, max_rows=1 << 25)
    kw = dict(c=cache(kv_heads=1), heads=64, qs=64 * 64)
    assert attend(b=b, os_=64 * 64, **kw) == cfz.CFZ_ERR_SHAPE
    assert select(b=b, bl=lists(q_block=1 << 25), **kw) == cfz.CFZ_ERR_SHAPE
    assert append(c=cache(kv_heads=128), b=batch(tokens=1 << 21, max_rows=1 << 21), ks=8192,
                  vs=8192) == cfz.CFZ_ERR_SHAPE
    assert cfz.cfz_last_error().endswith("work-groups (limit 2^23)")
    assert attend(b=batch(table_width=(1 << 25) + 1), max_kv=(1 << 30) + 1) == cfz.CFZ_ERR_SHAPE
    assert cfz.cfz_last_error().endswith("at most 2^30)")


def test_lists_count_whole_in_the_workspace():
    """The parts of a call with lists are counted by the lists' places, whatever max_kv is."""
    c, b = cache(), batch(table_width=64)
    need = [cfz._lib.cfz_kv8_attend_workspace_bytes(C.byref(c), C.byref(b), 2, kv,
                                                    C.byref(lists(count=4096, q_block=16)))
            for kv in (2, 2048)]
    assert need[0] == need[1] > 0


def test_share_plan():
    from diffusion_activation_residual_amd import cadence
    p = cadence.SharePlan(2, [40, 96, 33], 40, 32, device="cpu")
    assert (p.tokens, p.width, p.pages) == (169, 6, 12)
    assert p.table.tolist() == [[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11]]
    assert [s.tolist() for s in p.starts] == [[0, 0], [40, 40], [136, 136]]
    assert [o.tolist() for o in p.offsets] == [[0, 40, 80], [0, 96, 192], [0, 33, 66]]
    assert p.lengths.tolist() == [169, 169] and p.q_offsets.tolist() == [0, 40, 80]
    for bad in (dict(batch=0), dict(share_tokens=[]), dict(share_tokens=[3, 0]), dict(queries=0),
                dict(page_tokens=48), dict(count=0), dict(count=2, first=2, last=1),
                dict(count=1, q_block=0), dict(count=1, first=-1)):
        kw = dict(batch=1, share_tokens=[8], queries=1, page_tokens=32, device="cpu")
        with pytest.raises(ValueError):
            cadence.SharePlan(**{**kw, **bad})


def test_layer_attention_refusals():
    """Everything is checked before a stream is touched (none of these calls gets that far)."""
    from types import SimpleNamespace as N

    import torch

    from diffusion_activation_residual_amd import cadence
    plan = cadence.SharePlan(2, [8, 8], 4, 32, device="cpu")
    t, q = torch.zeros(16, 2, 64), torch.zeros(8, 2, 64)
    pool, share = N(page_tokens=32, pages=2), cadence.Share(t, t)
    good = dict(layers=[[share, share]], caches=[pool], q=[q], out=[q], streams=[])
    for bad in (dict(), dict(layers=[]), dict(out=[q, q]), dict(layers=[[share]]),
                dict(layers=[[share, cadence.Share(t[1:], t)]]),
                dict(layers=[[share, cadence.Share(t, t, receivers=(1, 2))]]),
                dict(layers=[[share, cadence.Share(t, t, codes=(t, t), scales=(t, t))]]),
                dict(q=[q[1:]]), dict(caches=[N(page_tokens=64, pages=2)]),
                dict(caches=[N(page_tokens=32, pages=1)])):
        with pytest.raises(ValueError):
            cadence.enqueue_layer_attention(plan, **{**good, **bad})
