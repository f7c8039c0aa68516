"""Host-side checks of include/cfz_block.h that need no GPU: exported functions, a header that stands on
its own, and refusals with the documented status before any device work (every call below fails
validation or is a no-op)."""
import ctypes as C
import os
import re
import shutil
import subprocess

import pytest

from diffusion_activation_residual_amd import block, cfz, kv8
from test_kv8_boundary_cpu import A, ODD, ref, rotation

lib = cfz._lib
HEADER = os.path.join(os.path.dirname(cfz.HEADER_PATH), "cfz_block.h")
NULL, SHAPE, UNSUP, ALIGN = (cfz.CFZ_ERR_NULL, cfz.CFZ_ERR_SHAPE, cfz.CFZ_ERR_UNSUPPORTED,
                             cfz.CFZ_ERR_ALIGN)
NAN, INF = float("nan"), float("inf")


def test_header_functions_are_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(cfz_[a-z_0-9]+)\s*\(", text))
    assert names == set(block._SIGNATURES)
    for name in names:
        assert hasattr(lib, name)


@pytest.mark.skipif(shutil.which("gcc") is None or shutil.which("g++") is None,
                    reason="gcc/g++ not available")
def test_header_is_self_contained_c_and_cxx_with_the_bindings_layout(tmp_path):
    """The structures' sizes and last members' places in C are the binding's."""
    structs = [s for s in vars(block).values() if isinstance(s, type) and issubclass(s, C.Structure)
               and s.__module__ == block.__name__] + [kv8.cfz_kv8_pages]
    lines = "".join(
        f'_Static_assert(sizeof({s.__name__}) == {C.sizeof(s)}, "{s.__name__}");\n'
        f'_Static_assert(offsetof({s.__name__}, {s._fields_[-1][0]}) == '
        f'{getattr(s, s._fields_[-1][0]).offset}, "{s.__name__}");\n' for s in structs)
    src = tmp_path / "inc.c"
    src.write_text('#include "cfz_block.h"\n#include <stddef.h>\n' + lines +
                   "int main(void) { return 0; }\n")
    cxx = tmp_path / "inc.cpp"
    cxx.write_text('#include "cfz_block.h"\nint main() { return 0; }\n')
    for comp, std, f in (("gcc", "-std=c11", src), ("g++", "-std=c++17", cxx)):
        r = subprocess.run([comp, std, "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                            os.path.dirname(HEADER), "-c", str(f), "-o", str(tmp_path / "o.o")],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


# ------------------------------------------------------------------ the norms

def norm(kind=1, eps=1e-6, weight=None, bias=None, dtype=0):
    return block.cfz_norm(kind, eps, weight, bias, dtype)


def items(data=A, stride=64, dtype=0):
    return block.cfz_item_rows(data, stride, dtype)


def residual(**kw):
    d = dict(tokens=4, cols=64, batch=1, offsets=None, x_dtype=0, y_dtype=0, x=A, x_stride=64, y=A,
             y_stride=64, r=A, r_stride=64, h=A, h_stride=64, gate_scale=1.0, gate=items(),
             scale=items(), shift=items(), after=norm(), before=norm())
    d.update(kw)
    a = block.cfz_residual()
    for k, v in d.items():
        setattr(a, k, v)
    return lib.cfz_residual_norm(C.byref(a), None)


WIDE = dict(cols=512, x_stride=512, y_stride=512, r_stride=512, h_stride=512, gate=items(stride=0),
            scale=items(stride=0), shift=items(stride=0))


@pytest.mark.parametrize("kw,status", [
    (dict(x_dtype=3), UNSUP), (dict(y_dtype=-1), UNSUP), (dict(x_dtype=1), UNSUP),
    (dict(x_dtype=0, y_dtype=2), UNSUP), (dict(cols=0), SHAPE), (dict(cols=12), SHAPE),
    (dict(cols=16392), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE),
    (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE), (dict(batch=3), SHAPE),
    (dict(offsets=A + 2), ALIGN), (dict(gate_scale=NAN), SHAPE), (dict(gate_scale=INF), SHAPE),
    (dict(gate=items(dtype=1)), UNSUP), (dict(gate=items(data=ODD)), ALIGN),
    (dict(scale=items(stride=32)), SHAPE), (dict(shift=items(stride=65)), SHAPE),
    (dict(scale=items(dtype=2, stride=66)), SHAPE), (dict(after=norm(kind=3)), UNSUP),
    (dict(before=norm(kind=-1)), UNSUP), (dict(before=norm(eps=-1.0)), SHAPE),
    (dict(before=norm(eps=NAN)), SHAPE), (dict(after=norm(eps=INF)), SHAPE),
    (dict(before=norm(bias=A)), UNSUP), (dict(before=norm(kind=0, weight=A)), UNSUP),
    (dict(after=norm(weight=A, dtype=1)), UNSUP), (dict(after=norm(weight=ODD)), ALIGN),
    (dict(x_stride=32), SHAPE), (dict(x_stride=68), SHAPE), (dict(x_stride=1 << 31), SHAPE),
    (dict(y_stride=8), SHAPE), (dict(r_stride=8), SHAPE), (dict(h_stride=65), SHAPE),
    (dict(x=None), NULL), (dict(r=None, h=None), NULL), (dict(y=None), NULL),
    (dict(y=None, gate=items(data=None)), NULL), (dict(x=ODD), ALIGN), (dict(h=ODD), ALIGN),
    (dict(r_stride=72), SHAPE), (dict(h_stride=72), SHAPE),
    (dict(cols=8192, tokens=1 << 23, x_stride=8192, y_stride=8192, r_stride=8192, h_stride=8192,
          gate=items(stride=0), scale=items(stride=0), shift=items(stride=0)), SHAPE),
    (dict(tokens=1 << 28), SHAPE), (dict(tokens=(1 << 28) - 32, x=None), NULL),
    (dict(WIDE, tokens=1 << 25), SHAPE), (dict(WIDE, tokens=(1 << 25) - 4, x=None), NULL),
    (dict(tokens=0, x=None, batch=5), cfz.CFZ_OK),
    (dict(tokens=0, x=None, y=None, r=None, h=None, gate=items()), cfz.CFZ_OK),
])
def test_norm_refusals(kw, status):
    assert residual(**kw) == status
    assert status == cfz.CFZ_OK or cfz.cfz_last_error()
    assert lib.cfz_residual_norm(None, None) == NULL


# ------------------------------------------------------------------ tables and rotation

def table(rows=4, positions=None, cos=A, sin=A, **kw):
    d = dict(rot_dim=64, axes=1, axis_dim=(64, 0, 0, 0), scaling=0, base=1e4, factor=1.0, trained=0.0,
             slow=1.0, fast=32.0, amplitude=1.0)
    d.update(kw)
    d["axis_dim"] = (C.c_int32 * 4)(*d["axis_dim"])
    return lib.cfz_rotation_table(C.byref(block.cfz_rotation_angles(**d)), rows, positions, cos, sin,
                                  None)


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), SHAPE), (dict(rot_dim=12, axis_dim=(12, 0, 0, 0)), SHAPE),
    (dict(rot_dim=264), SHAPE), (dict(axes=0), SHAPE), (dict(axes=5), SHAPE),
    (dict(scaling=4), UNSUP), (dict(scaling=-1), UNSUP), (dict(axis_dim=(32, 0, 0, 0)), SHAPE),
    (dict(axes=2, axis_dim=(61, 3, 0, 0), positions=A), SHAPE),
    (dict(axes=2, axis_dim=(64, 0, 0, 0), positions=A), SHAPE),
    (dict(axes=2, axis_dim=(62, 2, 0, 0), positions=A, scaling=2), SHAPE),
    (dict(axes=2, axis_dim=(32, 32, 0, 0)), NULL), (dict(base=1.0), SHAPE), (dict(base=NAN), SHAPE),
    (dict(factor=0.0), SHAPE), (dict(factor=INF), SHAPE), (dict(amplitude=0.0), SHAPE),
    (dict(amplitude=NAN), SHAPE), (dict(scaling=3), SHAPE), (dict(scaling=3, trained=INF), SHAPE),
    (dict(scaling=3, trained=9.0, slow=-1.0), SHAPE),
    (dict(scaling=3, trained=9.0, slow=2.0, fast=2.0), SHAPE), (dict(rows=-1), SHAPE),
    (dict(rows=1 << 31), SHAPE), (dict(rows=1 << 26), SHAPE), (dict(positions=A + 1), ALIGN),
    (dict(scaling=2, base=1e300, factor=1e300), SHAPE), (dict(cos=None), NULL), (dict(sin=ODD), ALIGN),
    (dict(rows=0, cos=None, sin=None), cfz.CFZ_OK),
])
def test_table_refusals(kw, status):
    assert table(**kw) == status
    assert lib.cfz_rotation_table(None, 1, None, A, A, None) == NULL


def rotate(count=1, dtype=0, dim=64, tokens=4, batch=1, offsets=A, starts=A, rot=rotation(), normed=1,
           eps=1e-6, **kw):
    d = dict(x=A, x_stride=128, out=A, out_stride=128, heads=2, weight=A, weight_dtype=0)
    d.update(kw)
    rows = (block.cfz_rotate_rows * 4)(*[block.cfz_rotate_rows(**d)] * 4)
    return lib.cfz_rotate(count, rows, dtype, dim, tokens, batch, offsets, starts, ref(rot), normed, eps,
                          None)


@pytest.mark.parametrize("kw,status", [
    (dict(count=0), SHAPE), (dict(count=5), SHAPE), (dict(dtype=3), UNSUP), (dict(dim=96), UNSUP),
    (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(batch=0), SHAPE),
    (dict(batch=65536), SHAPE), (dict(offsets=A + 2), ALIGN), (dict(starts=A + 2), ALIGN),
    (dict(batch=2, offsets=None), NULL), (dict(rot=None, normed=0, weight=None), NULL),
    (dict(normed=0), UNSUP), (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE),
    (dict(rot=rotation(rot_dim=4)), SHAPE), (dict(rot=rotation(rot_dim=72)), SHAPE),
    (dict(rot=rotation(table_rows=0)), SHAPE), (dict(rot=rotation(cos=None)), NULL),
    (dict(rot=rotation(sin=ODD)), ALIGN), (dict(rot=rotation(positions=A + 1)), ALIGN),
    (dict(heads=0), SHAPE), (dict(heads=1025, x_stride=1 << 17, out_stride=1 << 17), SHAPE),
    (dict(x_stride=120), SHAPE), (dict(x_stride=132), SHAPE), (dict(out_stride=64), SHAPE),
    (dict(weight_dtype=1), UNSUP), (dict(weight=ODD), ALIGN), (dict(x=None), NULL),
    (dict(out=None), NULL), (dict(x=ODD), ALIGN), (dict(out_stride=136), SHAPE),
    (dict(tokens=(1 << 31) - 1, heads=1024, x_stride=1 << 16, out_stride=1 << 16), SHAPE),
    (dict(tokens=0, x=None, out=None), cfz.CFZ_OK),
])
def test_rotate_refusals(kw, status):
    assert rotate(**kw) == status
    assert lib.cfz_rotate(1, None, 0, 64, 4, 1, None, None, None, 1, 0.0, None) == NULL


# ------------------------------------------------------------------ adapters

def adapters(tokens=4, batch=1, offsets=A, ids=A, max_rows=4, x=A, xs=64, y=A, ys=64, out=A, os_=64,
             y_dtype=0, ws=A, n=1 << 20, **kw):
    d = dict(adapters=2, slices=2, rank=8, cols_in=64, slice_cols=(48, 16, 0, 0), dtype=0, a=A, b=A,
             scale=A)
    d.update(kw)
    d["slice_cols"] = (C.c_int32 * 4)(*d["slice_cols"])
    w = block.cfz_adapters(**d)
    size = lib.cfz_adapters_workspace_bytes(C.byref(w), tokens, batch)
    return lib.cfz_adapters_add(C.byref(w), tokens, batch, offsets, ids, max_rows, x, xs, y, ys, out, os_,
                                y_dtype, ws, n, None), size


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUP), (dict(adapters=0), SHAPE), (dict(adapters=(1 << 20) + 1), SHAPE),
    (dict(slices=0), SHAPE), (dict(slices=5), SHAPE), (dict(rank=4), SHAPE), (dict(rank=12), SHAPE),
    (dict(rank=136), SHAPE),
    (dict(cols_in=0), SHAPE), (dict(cols_in=60), SHAPE), (dict(cols_in=(1 << 20) + 8), SHAPE),
    (dict(slice_cols=(48, 8, 0, 0)), SHAPE), (dict(slice_cols=(48, 0, 0, 0)), SHAPE),
    (dict(slice_cols=(1 << 20, 16, 0, 0)), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(tokens=1 << 31), SHAPE), (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE),
    (dict(y_dtype=1), UNSUP), (dict(max_rows=-1), SHAPE), (dict(max_rows=1 << 31), SHAPE),
    (dict(xs=32), SHAPE), (dict(xs=68), SHAPE), (dict(ys=48), SHAPE), (dict(os_=65), SHAPE),
    (dict(os_=72), SHAPE), (dict(a=None), NULL), (dict(b=None), NULL), (dict(offsets=None), NULL),
    (dict(ids=None), NULL), (dict(x=None), NULL), (dict(y=None), NULL), (dict(out=None), NULL),
    (dict(a=ODD), ALIGN), (dict(x=ODD), ALIGN), (dict(ids=A + 2), ALIGN), (dict(scale=A + 1), ALIGN),
    (dict(ws=None), cfz.CFZ_ERR_WORKSPACE), (dict(n=100), cfz.CFZ_ERR_WORKSPACE),
    (dict(ws=A + 16), ALIGN),
    (dict(tokens=(1 << 31) - 1, slices=1, slice_cols=(1 << 20, 0, 0, 0), ys=1 << 20, os_=1 << 20),
     SHAPE),
    (dict(tokens=0, x=None), cfz.CFZ_OK), (dict(batch=0, ids=None), cfz.CFZ_OK),
    (dict(max_rows=0, x=None), cfz.CFZ_OK),
])
def test_adapter_refusals(kw, status):
    assert adapters(**kw)[0] == status
    assert lib.cfz_adapters_add(None, 0, 0, None, None, 0, None, 0, None, 0, None, 0, 0, None, 0,
                                None) == NULL


@pytest.mark.parametrize("first,count,a,rows,status", [
    (-1, 1, A, A, SHAPE), (0, -1, A, A, SHAPE), (2, 1, A, A, SHAPE), (1 << 30, 1 << 30, A, A, SHAPE),
    (0, 1, None, A, NULL), (0, 1, A, None, NULL), (0, 1, ODD, A, ALIGN), (0, 1, A, ODD, ALIGN),
    (2, 0, None, None, cfz.CFZ_OK),
])
def test_adapter_layout_refusals(first, count, a, rows, status):
    w = block.cfz_adapters(2, 1, 8, 64, (C.c_int32 * 4)(64), 0, a, None, None)
    assert lib.cfz_adapters_put(C.byref(w), first, count, rows, None) == status
    assert lib.cfz_adapters_put(None, 0, 0, None, None) == NULL
    assert lib.cfz_adapters_a_bytes(C.byref(w)) == 2 * 16 * 128 * 2
    w.cols_in, w.rank = 40, 24
    assert lib.cfz_adapters_a_bytes(C.byref(w)) == 2 * 32 * 128 * 2
    w.rank = 7
    assert lib.cfz_adapters_a_bytes(C.byref(w)) == 0


def test_adapter_workspaces():
    """A row of all slices' low-rank values and a number for each slice, for each token; nothing for no
    tokens or sequences."""
    assert adapters()[1] == 4 * (16 + 2) * 4
    assert adapters(tokens=0)[1] == adapters(batch=0)[1] == adapters(rank=7)[1] == 0
    assert adapters(cols_in=4096, xs=4096)[1] == 4 * (16 + 2) * 4
