"""Binding over ``include/cfz_block.h``: what lies between a transformer layer's residual stream and
the 8-bit K/V cache (``kv8``).

``residual_norm`` adds a block's gated output to the stream and normalises the sum for the next
block; ``rotation_table`` makes the tables of a ``kv8.Rotation`` and ``rotate`` turns queries and
keys by them; ``Adapters`` adds the low-rank adapters of many requests to a projection that they
share.  Argument marshalling only: every step runs in the library's HIP kernels.  Because it
sees tensor sizes, which the C ABI cannot, this module refuses (``ValueError`` or ``TypeError``,
before any device work) tensors that do not fit the call.  Work is queued on ``stream`` (default:
the current one of the tensors' device); with another stream than the current one the caller orders
the tensors' other uses.  Nothing is recorded for autograd: results carry no gradient."""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from typing import Optional

import torch

from . import cfz, kv8
from .cfz import CFZ_ERR_NULL, CFZ_OK, CfzError
from .kv8 import _REALS, _empty_on, _fit, _held, _ints, _queue, cfz_kv8_rotation

NORMS = {"none": 0, "rms": 1, "layer": 2}
SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


class cfz_norm(C.Structure):
    _fields_ = [("kind", C.c_int32), ("eps", C.c_float), ("weight", C.c_void_p),
                ("bias", C.c_void_p), ("dtype", C.c_int32)]


class cfz_item_rows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("stride", C.c_int64), ("dtype", C.c_int32)]


class cfz_residual(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("cols", C.c_int32), ("batch", C.c_int32),
                ("offsets", C.c_void_p), ("x_dtype", C.c_int32), ("y_dtype", C.c_int32),
                ("x", C.c_void_p), ("x_stride", C.c_int64), ("y", C.c_void_p),
                ("y_stride", C.c_int64), ("r", C.c_void_p), ("r_stride", C.c_int64),
                ("h", C.c_void_p), ("h_stride", C.c_int64), ("gate_scale", C.c_float),
                ("gate", cfz_item_rows), ("scale", cfz_item_rows), ("shift", cfz_item_rows),
                ("after", cfz_norm), ("before", cfz_norm)]


class cfz_rotation_angles(C.Structure):
    _fields_ = [("rot_dim", C.c_int32), ("axes", C.c_int32), ("axis_dim", C.c_int32 * 4),
                ("scaling", C.c_int32), ("base", C.c_double), ("factor", C.c_double),
                ("trained", C.c_double), ("slow", C.c_double), ("fast", C.c_double),
                ("amplitude", C.c_double)]


class cfz_rotate_rows(C.Structure):
    _fields_ = [("x", C.c_void_p), ("x_stride", C.c_int64), ("out", C.c_void_p),
                ("out_stride", C.c_int64), ("heads", C.c_int32), ("weight", C.c_void_p),
                ("weight_dtype", C.c_int32)]


class cfz_adapters(C.Structure):
    _fields_ = [("adapters", C.c_int32), ("slices", C.c_int32), ("rank", C.c_int32),
                ("cols_in", C.c_int32), ("slice_cols", C.c_int32 * 4), ("dtype", C.c_int32),
                ("a", C.c_void_p), ("b", C.c_void_p), ("scale", C.c_void_p)]


_p, _i64, _i32, _f32 = C.c_void_p, C.c_int64, C.c_int32, C.c_float
_SIGNATURES = {
    "cfz_residual_norm": ([C.POINTER(cfz_residual), _p], _i32),
    "cfz_rotation_table": ([C.POINTER(cfz_rotation_angles), _i64, _p, _p, _p, _p], _i32),
    "cfz_rotate": ([_i32, C.POINTER(cfz_rotate_rows), _i32, _i32, _i64, _i32, _p, _p,
                    C.POINTER(cfz_kv8_rotation), _i32, _f32, _p], _i32),
    "cfz_adapters_a_bytes": ([C.POINTER(cfz_adapters)], C.c_size_t),
    "cfz_adapters_put": ([C.POINTER(cfz_adapters), _i32, _i32, _p, _p], _i32),
    "cfz_adapters_add": ([C.POINTER(cfz_adapters), _i64, _i32, _p, _p, _i64, _p, _i64, _p, _i64,
                          _p, _i64, _i32, _p, C.c_size_t, _p], _i32),
    "cfz_adapters_workspace_bytes": ([C.POINTER(cfz_adapters), _i64, _i32], C.c_size_t),
}
_lib = cfz._lib
for _name, (_args, _res) in _SIGNATURES.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _res


def _device(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what}: libcfz takes device tensors")
    return t.device


def _as_stream(stream, device):
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream, device)
    return torch.cuda.current_stream(device) if stream is None else stream


def _matrix(t, shape, dtypes, device, what):
    """Row stride of a [rows, cols] tensor with dense rows."""
    stride = t.stride()
    if t.dtype in dtypes and t.device == device and t.shape == shape and stride[1] == 1:
        return stride[0] if shape[0] > 1 else shape[1]
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: {t.dtype}, expected one of {dtypes}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    rows, cols = shape
    if t.numel() and cols > 1:
        raise ValueError(f"{what}: a row's values must lie side by side (strides {stride})")
    return stride[0] if rows > 1 else cols


def _vector(t, size, dtype, device, what):
    """Address and type of a weight."""
    if t.dtype == dtype and t.device == device and t.shape == (size,) and t.is_contiguous():
        return t.data_ptr(), _REALS[dtype]
    if t.dtype != dtype and t.dtype != torch.float32:
        raise TypeError(f"{what}: {t.dtype}, expected {dtype} or fp32")
    if t.device != device or t.shape != (size,) or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor of {size} values on {device}")
    return t.data_ptr(), _REALS[t.dtype]


@dataclass
class Norm:
    """A norm over a row's columns: ``kind`` "rms" or "layer", ``weight`` and (layer) ``bias`` [cols],
    fp32 or of the type of the rows that leave the norm, or None."""

    kind: str = "rms"
    eps: float = 1e-6
    weight: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None


def _norm(norm, cols, dtype, device, what):
    if norm.kind not in NORMS:
        raise ValueError(f"{what}: kind = {norm.kind!r}, one of {sorted(NORMS)}")
    weight = bias = None
    kind = _REALS[dtype]
    if norm.weight is not None:
        weight, kind = _vector(norm.weight, cols, dtype, device, what + ".weight")
    if norm.bias is not None:
        bias, other = _vector(norm.bias, cols, dtype, device, what + ".bias")
        if weight is not None and other != kind:
            raise TypeError(f"{what}: weight and bias must be of one type")
        kind = other
    return cfz_norm(NORMS[norm.kind], norm.eps, weight, bias, kind)


def _items(t, batch, cols, dtype, device, what):
    """[batch, cols] rows (possibly apart, as chunks of one projection are), [1, cols] or [cols]."""
    if t.dim() == 1:
        t = t[None]
    if t.dim() != 2 or t.shape[0] not in (1, batch):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected [{batch}, {cols}]")
    stride = _matrix(t, (t.shape[0], cols), (dtype, torch.float32), device, what)
    return cfz_item_rows(t.data_ptr(), 0 if t.shape[0] == 1 else stride, _REALS[t.dtype])


def residual_norm(x, y=None, *, before=None, after=None, gate=None, gate_scale=1.0, scale=None,
                  shift=None, offsets=None, batch=None, dtype=None, out=None, normed=None,
                  stream=None):
    """One step along the residual stream x [tokens, cols] (bf16, fp16 or fp32), returning (r, h):

        r = x + gate_scale * gate * after(y)          in x's type
        h = before(r) * (1 + scale) + shift           in y's type

    y [tokens, cols]: the block's output, of x's type or, beside an fp32 stream, bf16 or fp16; None
    takes r = x (and h is of ``dtype``, by default x's).  ``before`` and ``after`` are ``Norm``
    or None; without ``before``, scale and shift there is no h (None).  gate, scale and shift: a row
    for each item of the batch ([batch, cols]; rows may lie apart), or one for all.  ``offsets``
    (int32 [batch + 1]) gives the items' rows; rows of no item are left alone (unset, where r and h
    are allocated here).  Without it the items have equally many rows.  ``out`` may be x and
    ``normed`` may be y: in place."""
    a, device, out, normed = _residual(x, y, before, after, gate, gate_scale, scale, shift, offsets,
                                       batch, dtype, out, normed, stream)
    _queue(_lib.cfz_residual_norm, device, stream, C.byref(a))
    return out, normed


def check_residual_norm(x, y=None, *, out, normed, before=None, after=None, gate=None, gate_scale=1.0,
                        scale=None, shift=None, offsets=None, batch=None, dtype=None):
    """Raises where ``residual_norm`` would refuse these arguments (out and normed: given, or None where
    the call would leave them out); queues nothing."""
    a, *_ = _residual(x, y, before, after, gate, gate_scale, scale, shift, offsets, batch, dtype, out,
                      normed, None)
    if a.x % 16 if a.x else 0:
        raise ValueError(f"x: {a.x:#x}, expected 16-byte alignment")
    if out is not None and a.r == a.x and a.r_stride != a.x_stride:
        raise ValueError("in place, the strides must be the same")
    a.x = None  # (the last thing that the library asks for, after these two)
    missing = not (a.r or a.h) or not a.y and (a.gate.data or a.after.kind)
    status = _lib.cfz_residual_norm(C.byref(a), None)
    if status != (CFZ_OK if a.tokens == 0 else CFZ_ERR_NULL) or (missing and a.tokens):
        raise CfzError(status, "cfz_residual_norm")


def _residual(x, y, before, after, gate, gate_scale, scale, shift, offsets, batch, dtype, out, normed,
              stream):
    """The call's arguments, checked as far as the library does not see them, and its results."""
    device = _device(x, "x")
    if x.dim() != 2 or x.dtype not in _REALS:
        raise ValueError(f"x: {x.dtype} {tuple(x.shape)}, expected bf16, fp16 or fp32 [tokens, cols]")
    shape = tokens, cols = x.shape
    if dtype is None:
        dtype = x.dtype if y is None else y.dtype
    if dtype not in _REALS or (y is not None and y.dtype != dtype):
        raise TypeError(f"dtype = {dtype}: bf16, fp16 or fp32, and y's")
    if offsets is not None:
        batch = offsets.numel() - 1
    elif batch is None:
        batch = max([1] + [t.shape[0] for t in (gate, scale, shift) if t is not None and t.dim() == 2])
    if not (cols < 1 << 31 and -(1 << 31) <= batch < 1 << 31):
        _fit(32, cols=cols, batch=batch)
    a = cfz_residual()
    a.tokens, a.cols, a.batch = tokens, cols, batch
    if offsets is not None:
        a.offsets = _ints(offsets, (batch + 1,), device, "offsets")
    a.x_dtype, a.y_dtype = _REALS[x.dtype], _REALS[dtype]
    a.x, a.x_stride = x.data_ptr(), _matrix(x, shape, _REALS, device, "x")
    if y is not None:
        a.y, a.y_stride = y.data_ptr(), _matrix(y, shape, _REALS, device, "y")
    a.gate_scale = gate_scale
    if gate is not None:
        a.gate = _items(gate, batch, cols, dtype, device, "gate")
    if scale is not None:
        a.scale = _items(scale, batch, cols, dtype, device, "scale")
    if shift is not None:
        a.shift = _items(shift, batch, cols, dtype, device, "shift")
    if after is not None:
        a.after = _norm(after, cols, dtype, device, "after")
    if before is not None:
        a.before = _norm(before, cols, dtype, device, "before")
    if out is not None:
        a.r, a.r_stride = out.data_ptr(), _matrix(out, shape, (x.dtype,), device, "out")
    elif y is not None:
        out = _empty_on(device, stream, shape, x.dtype)
        a.r, a.r_stride = out.data_ptr(), cols
    else:
        out = x  # (nothing changes: no copy is made)
    if normed is not None:
        a.h, a.h_stride = normed.data_ptr(), _matrix(normed, shape, (dtype,), device, "normed")
    elif before is not None or scale is not None or shift is not None:
        normed = _empty_on(device, stream, shape, dtype)
        a.h, a.h_stride = normed.data_ptr(), cols
    return a, device, out, normed


def rotation_table(rot_dim, rows=None, positions=None, axis_dims=None, base=10000.0, scaling="none",
                   factor=1.0, trained=0, slow=1.0, fast=32.0, amplitude=1.0, interleaved=False,
                   device="cuda", stream=None):
    """A ``kv8.Rotation`` whose row t holds the cosines and sines (times ``amplitude``) of position
    t, for t < ``rows``, or of ``positions[t]`` (int32 [rows] or [rows, axes]).  ``axis_dims`` deals
    the rot_dim dimensions out to several axes (frame, row, column), by default one.  Pair i of an
    axis with d dimensions turns by base ** (-2 i / d) a position, stretched over contexts ``factor``
    times as long by ``scaling``: "linear" (slower by the factor), "base" (a larger base: the fastest
    pair as before, the slowest slower by the factor) or "parts" (pairs that turn more than ``fast``
    times over the ``trained`` length as before, those that turn less than ``slow`` times slower by
    the factor, a ramp between)."""
    if scaling not in SCALINGS:
        raise ValueError(f"scaling = {scaling!r}, one of {sorted(SCALINGS)}")
    axis_dims = [rot_dim] if axis_dims is None else list(axis_dims)
    if not 1 <= len(axis_dims) <= 4:
        raise ValueError(f"axis_dims = {axis_dims}: one to four")
    if positions is not None:
        device = _device(positions, "positions")
        shape = (positions.shape[0],) if positions.dim() == 1 and len(axis_dims) == 1 else \
            (positions.shape[0] if positions.dim() else 0, len(axis_dims))
        _ints(positions, shape, device, "positions")
        if rows is not None and rows != shape[0]:
            raise ValueError(f"rows = {rows} with {shape[0]} positions")
        rows = shape[0]
    elif rows is None:
        raise ValueError("rows or positions")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"device = {device}: libcfz writes device tensors")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    _fit(32, rot_dim=rot_dim, **{f"axis_{i}": d for i, d in enumerate(axis_dims)})
    _fit(64, rows=rows)
    if rows < 0 or rot_dim < 0:
        raise ValueError(f"rows = {rows}, rot_dim = {rot_dim}")
    angles = cfz_rotation_angles(rot_dim, len(axis_dims), (C.c_int32 * 4)(*axis_dims),
                                 SCALINGS[scaling], base, factor, trained, slow, fast, amplitude)
    where = None if positions is None else positions.data_ptr()
    # (the tables are the last thing that the library asks for: nothing is allocated for what it refuses)
    status = _lib.cfz_rotation_table(C.byref(angles), rows, where, None, None, None)
    if status != (CFZ_OK if rows == 0 else CFZ_ERR_NULL):
        raise CfzError(status, "cfz_rotation_table")
    cos, sin = (_empty_on(device, stream, (rows, rot_dim // 2), torch.float32) for _ in range(2))
    _queue(_lib.cfz_rotation_table, device, stream, C.byref(angles), rows, where, cos.data_ptr(),
           sin.data_ptr())
    return kv8.Rotation(cos, sin, interleaved=interleaved)


def rotate(tensors, rotation, offsets=None, starts=None, weights=None, eps=1e-6, normed=None,
           outs=None, stream=None):
    """Norm and rotation of each head of up to four tensors [tokens, heads, head_dim] (bf16, fp16 or
    fp32; views of one projection, say its queries and keys), in one launch: a list of results,
    dense or written to ``outs`` (which may be the tensors themselves; None: allocated).

    A head becomes x / sqrt(mean(x ** 2) + eps) * weight where ``weights`` gives one weight
    [head_dim] (or None) for each tensor (``normed=True``: without weights), and is then turned by
    ``rotation`` (None: the norm alone).  Row i of sequence b (rows offsets[b] .. offsets[b + 1] - 1;
    no offsets: all rows are one sequence) is at position starts[b] + i, where ``rotation`` names no
    positions.  Keys turned here are appended to a cache without a rotation."""
    return _rotate(_queue, tensors, rotation, offsets, starts, weights, eps, normed, outs, stream)


def check_rotate(tensors, rotation, offsets=None, starts=None, weights=None, eps=1e-6, normed=None):
    """Raises where ``rotate`` would refuse these arguments (its results allocated by itself); queues
    and allocates nothing."""
    _rotate(_ask, tensors, rotation, offsets, starts, weights, eps, normed, None, None)


def _ask(call, device, stream, count, rows, *args):
    """A rotation that is only checked: its tensors are left out, the last thing that the library asks for."""
    for i, row in enumerate(rows):
        if row.x % 16 if row.x else 0:
            raise ValueError(f"tensors[{i}]: {row.x:#x}, expected 16-byte alignment")
        row.x = None
    tokens, rotation, normed = args[2], args[6], args[7]
    nothing = rotation is None and not normed  # (asked for before)
    status = call(count, rows, *args, None)
    if nothing or status != (CFZ_OK if tokens == 0 else CFZ_ERR_NULL):
        raise CfzError(status, call.__name__)


def _rotate(queue, tensors, rotation, offsets, starts, weights, eps, normed, outs, stream):
    tensors = list(tensors)
    if not 1 <= len(tensors) <= 4:
        raise ValueError(f"{len(tensors)} tensors: one to four")
    first = tensors[0]
    device = _device(first, "tensors[0]")
    if first.dim() != 3 or first.dtype not in _REALS:
        raise ValueError(f"tensors[0]: {first.dtype} {tuple(first.shape)}, expected bf16, fp16 or "
                         "fp32 [tokens, heads, head_dim]")
    tokens, dim, dtype = first.shape[0], first.shape[2], first.dtype
    if normed is None:
        normed = weights is not None
    if weights is None:
        weights = [None] * len(tensors)
    if len(weights) != len(tensors) or (outs is not None and len(outs) != len(tensors)):
        raise ValueError(f"{len(tensors)} tensors, {len(weights)} weights and "
                         f"{'no' if outs is None else len(outs)} outs")
    batch = 1 if offsets is None else offsets.numel() - 1
    args = (cfz_rotate_rows * len(tensors))()
    results = []
    for i, (t, w) in enumerate(zip(tensors, weights)):
        if t.dtype != dtype or t.dim() != 3 or t.shape[0] != tokens:
            raise ValueError(f"tensors[{i}]: {t.dtype} {tuple(t.shape)}, expected {dtype} [{tokens}, "
                             f"heads, {dim}]")
        heads = t.shape[1]
        stride = kv8._rows(t, heads, dim, device, f"tensors[{i}]")
        out, out_stride = None if outs is None else outs[i], heads * dim
        if out is None:
            if queue is not _ask:
                out = _empty_on(device, stream, (tokens, heads, dim), dtype)
        else:
            if out.dtype != dtype or out.shape != t.shape:
                raise ValueError(f"outs[{i}]: {out.dtype} {tuple(out.shape)}, expected {dtype} "
                                 f"{tuple(t.shape)}")
            out_stride = kv8._rows(out, heads, dim, device, f"outs[{i}]")
        if heads >= 1 << 31:
            _fit(32, heads=heads)
        row = args[i]
        row.x, row.x_stride, row.out_stride = t.data_ptr(), stride, out_stride
        row.out = None if out is None else out.data_ptr()
        row.heads = heads
        if w is not None:
            row.weight, row.weight_dtype = _vector(w, dim, dtype, device, f"weights[{i}]")
        results.append(out)
    queue(_lib.cfz_rotate, device, stream, len(tensors), args, _REALS[dtype], dim, tokens, batch,
          None if offsets is None else _ints(offsets, (batch + 1,), device, "offsets"),
          None if starts is None else _ints(starts, (batch,), device, "starts"),
          kv8._rotation(rotation, tokens, device), bool(normed), eps)
    return results


class Adapters:
    """Low-rank adapters of one projection, from ``a`` [adapters, slices * rank, cols_in] and ``b``
    [adapters, cols_out, rank], bf16 or fp16, and ``scale`` [adapters] fp32 or None (1).  ``slices``: how
    many parts of equal width the projection's columns have, or a list of their widths (query,
    key and value of one fused projection); part i is met by rows i * rank .. (i + 1) * rank - 1 of a.
    rank: a multiple of 8 up to 128; adapters of a lower one are filled up with zeros.

    a is copied into the layout that the kernels read; b and scale are used as they are.  ``put``
    replaces adapters in place (a pool that requests bring theirs to).  The calls know all three by their
    addresses: another tensor in their place is refused (ValueError)."""

    a, b, scale = map(_held, ("a", "b", "scale"))

    def __init__(self, a, b, scale=None, slices=1, stream=None):
        self.device = _device(a, "a")
        if a.dim() != 3 or b.dim() != 3 or a.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"a: {a.dtype} {tuple(a.shape)}, b: {tuple(b.shape)}, expected bf16 or "
                             "fp16 [adapters, slices * rank, cols_in] and [adapters, cols_out, rank]")
        count, cols_out, rank = b.shape
        if a.shape[0] != count:
            raise ValueError(f"a has {a.shape[0]} adapters, b {count}")
        if isinstance(slices, int):
            if slices < 1 or cols_out % slices:
                raise ValueError(f"slices = {slices} of {cols_out} columns")
            slices = [cols_out // slices] * slices
        slices = list(slices)
        if not 1 <= len(slices) <= 4 or sum(slices) != cols_out or min(slices) < 1:
            raise ValueError(f"slices = {slices} of {cols_out} columns")
        if b.dtype != a.dtype or b.device != self.device or not b.is_contiguous():
            raise ValueError("b: must be contiguous, of a's type and on its device")
        if scale is not None and (scale.dtype != torch.float32 or scale.shape != (count,) or
                                  scale.device != self.device or not scale.is_contiguous()):
            raise ValueError(f"scale: expected a contiguous fp32 tensor of {count} values")
        _fit(32, adapters=count, rank=rank, cols_in=a.shape[2], cols_out=cols_out)
        self.b, self.scale, self.slices, self.count = b, scale, slices, count
        self.rank, self.cols_in, self.cols_out, self.dtype = rank, a.shape[2], cols_out, a.dtype
        self.desc = cfz_adapters(count, len(slices), rank, self.cols_in, (C.c_int32 * 4)(*slices),
                                 _REALS[a.dtype], None, b.data_ptr(),
                                 None if scale is None else scale.data_ptr())
        self._ref = C.byref(self.desc)
        need = _lib.cfz_adapters_a_bytes(self._ref)
        if need == 0:  # (the call below says why)
            _queue(_lib.cfz_adapters_put, self.device, stream, self._ref, 0, 0, None)
        self.a = _empty_on(self.device, stream, need, torch.uint8)
        self.desc.a = self.a.data_ptr()
        self.put(0, a, stream=stream)

    def put(self, first, a, b=None, scale=None, stream=None):
        """Adapters first .. first + n - 1 become ``a`` [n, slices * rank, cols_in], with ``b`` [n,
        cols_out, rank] and ``scale`` (n values) copied into theirs where given."""
        shape = (a.shape[0], len(self.slices) * self.rank, self.cols_in)
        if a.dtype != self.dtype or a.shape != shape or a.device != self.device or \
                not a.is_contiguous():
            raise ValueError(f"a: {a.dtype} {tuple(a.shape)}, expected a contiguous {self.dtype} tensor "
                             f"{shape} on {self.device}")
        n = shape[0]
        if not 0 <= first <= self.count - n:
            raise ValueError(f"adapters {first} .. {first + n - 1} of {self.count}")
        if b is not None and (b.shape != (n, self.cols_out, self.rank) or b.dtype != self.dtype):
            raise ValueError(f"b: {b.dtype} {tuple(b.shape)}, expected {self.dtype} "
                             f"{(n, self.cols_out, self.rank)}")
        if scale is not None and (self.scale is None or scale.shape != (n,)):
            raise ValueError(f"scale: shape {tuple(scale.shape)}, expected ({n},) beside held scales")
        _queue(_lib.cfz_adapters_put, self.device, stream, self._ref, first, n, a.data_ptr())
        for held, new in ((self.b, b), (self.scale, scale)):
            if new is not None:
                with torch.cuda.stream(_as_stream(stream, self.device)), torch.inference_mode():
                    held[first:first + n].copy_(new)

    def add(self, x, y, ids, offsets, max_rows, out=None, workspace=None, stream=None):
        """y + scale * (x a^T) b^T for each sequence's own adapter: x [tokens, cols_in], y [tokens,
        cols_out] (the shared projection's rows, of x's type or fp32), ``ids`` [batch] int32 (-1: no
        adapter), ``offsets`` [batch + 1] int32 the sequences' rows, at most ``max_rows`` each.
        ``out`` may be y; without it the result is allocated (rows of no sequence are then left
        unset)."""
        if x.dim() != 2 or y.dim() != 2:
            raise ValueError(f"x {tuple(x.shape)}, y {tuple(y.shape)}: expected [tokens, cols]")
        tokens, batch = x.shape[0], ids.numel()
        xs = _matrix(x, (tokens, self.cols_in), (self.dtype,), self.device, "x")
        ys = _matrix(y, (tokens, self.cols_out), (self.dtype, torch.float32), self.device, "y")
        if not (batch < 1 << 31 and -(1 << 63) <= max_rows < 1 << 63):
            _fit(32, batch=batch)
            _fit(64, max_rows=max_rows)
        need = _lib.cfz_adapters_workspace_bytes(self._ref, tokens, batch)
        if out is None:
            out, os = _empty_on(self.device, stream, y.shape, y.dtype), self.cols_out
        else:
            os = _matrix(out, y.shape, (y.dtype,), self.device, "out")
        if workspace is None:
            workspace = _empty_on(self.device, stream, need, torch.uint8)
        elif workspace.device == self.device and workspace.is_contiguous():
            need = workspace.numel() * workspace.element_size()
        else:
            raise ValueError("workspace: must be contiguous and on the adapters' device")
        _queue(_lib.cfz_adapters_add, self.device, stream, self._ref, tokens, batch,
               _ints(offsets, (batch + 1,), self.device, "offsets"),
               _ints(ids, (batch,), self.device, "ids"), max_rows, x.data_ptr(), xs, y.data_ptr(), ys,
               out.data_ptr(), os, _REALS[y.dtype], workspace.data_ptr(), need)
        return out
