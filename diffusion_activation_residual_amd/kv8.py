"""Binding over libcfz's 8-bit paged K/V cache (``include/cfz_kv8.h``): argument marshalling and
``Cache``, which holds a pool's buffers in torch tensors.

What a receiver rebuilds with the codec -- one layer's K and V of another device's share -- is
appended to such a cache (straight from the receiver's fp32 base, if wanted), and the device's
own queries attend over all shares.  Every step runs in the library's HIP kernels.  Because it sees
tensor sizes, which the C ABI cannot, this module refuses (``ValueError`` or ``TypeError``,
before any device work) tensors that do not fit the call."""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from typing import Optional

import torch

from . import cfz
from .cfz import CFZ_ERR_NULL, CFZ_OK, CfzError

CFZ_KV8_INT8, CFZ_KV8_E4M3 = 0, 1
CFZ_KV8_BF16, CFZ_KV8_F16, CFZ_KV8_F32 = 0, 1, 2
FORMATS = {"int8": CFZ_KV8_INT8, "e4m3": CFZ_KV8_E4M3}
_CODES = {torch.int8: CFZ_KV8_INT8, torch.float8_e4m3fn: CFZ_KV8_E4M3}
_REALS = {torch.bfloat16: CFZ_KV8_BF16, torch.float16: CFZ_KV8_F16, torch.float32: CFZ_KV8_F32}


class cfz_kv8_cache(C.Structure):
    _fields_ = [("pages", C.c_int64), ("kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("page_tokens", C.c_int32), ("format", C.c_int32), ("k", C.c_void_p),
                ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("k_mean", C.c_void_p)]


class cfz_kv8_batch(C.Structure):
    _fields_ = [("batch", C.c_int32), ("table_width", C.c_int32), ("page_table", C.c_void_p),
                ("offsets", C.c_void_p), ("lengths", C.c_void_p), ("tokens", C.c_int64),
                ("max_rows", C.c_int64)]


class cfz_kv8_rotation(C.Structure):
    _fields_ = [("cos", C.c_void_p), ("sin", C.c_void_p), ("positions", C.c_void_p),
                ("table_rows", C.c_int64), ("rot_dim", C.c_int32), ("interleaved", C.c_int32)]


class cfz_kv8_blocks(C.Structure):
    _fields_ = [("blocks", C.c_void_p), ("count", C.c_int32), ("q_block", C.c_int32)]


class cfz_kv8_pages(C.Structure):
    _fields_ = [("pages", C.c_int64), ("batch", C.c_int32), ("table_width", C.c_int32),
                ("page_tokens", C.c_int32), ("page_table", C.c_void_p), ("lengths", C.c_void_p),
                ("refs", C.c_void_p)]


_p, _i64, _i32, _sz = C.c_void_p, C.c_int64, C.c_int32, C.c_size_t
_cache, _batch = C.POINTER(cfz_kv8_cache), C.POINTER(cfz_kv8_batch)
_blocks, _pages = C.POINTER(cfz_kv8_blocks), C.POINTER(cfz_kv8_pages)
_SIGNATURES = {
    "cfz_kv8_append": ([_cache, _batch, _i32, _p, _p, _i64, _i64, C.POINTER(cfz_kv8_rotation), _p],
                       _i32),
    "cfz_kv8_gather": ([_cache, _batch, _i32, _p, _p, _p], _i32),
    "cfz_kv8_attend": ([_cache, _batch, _i32, _p, _i64, _i32, _i32, C.c_float, _i64, _blocks, _p,
                        _i64, _p, _p, _sz, _p], _i32),
    "cfz_kv8_attend_workspace_bytes": ([_cache, _batch, _i32, _i64, _blocks], _sz),
    "cfz_kv8_select": ([_cache, _batch, _i32, _p, _i64, _i32, _i32, _i64, _i32, _i32, _blocks, _p,
                        _sz, _p], _i32),
    "cfz_kv8_select_workspace_bytes": ([_cache, _batch, _i64, _blocks], _sz),
    "cfz_kv8_free": ([_pages, _i32, _p, _p, _p], _i32),
    "cfz_kv8_fork": ([_pages, _i32, _p, _p, _p], _i32),
    "cfz_kv8_reserve": ([_pages, _p, _i64, _p, _p, _p, _p, _sz, _p], _i32),
    "cfz_kv8_reserve_rows": ([_pages, _p, _i64, _p, _p, _p, _p, _p, _sz, _p], _i32),
    "cfz_kv8_reserve_workspace_bytes": ([_pages, _i64], _sz),
    "cfz_kv8_compact": ([_pages, _p, _p, _p, _p, _p, _sz, _p], _i32),
    "cfz_kv8_compact_workspace_bytes": ([_pages], _sz),
    "cfz_kv8_copy": ([_cache, _cache, _i64, _p, _p, _p, _p], _i32),
}
_lib = cfz._lib
for _name, (_args, _res) in _SIGNATURES.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _res


@dataclass
class Rotation:
    """The rotation of appended keys: ``cos`` and ``sin`` [rows, rot_dim / 2] fp32, pair i being
    (i, i + rot_dim / 2) or, interleaved, (2 i, 2 i + 1); ``positions`` (int32, one per token
    row) picks the rows, by default the token's index in its sequence."""

    cos: torch.Tensor
    sin: torch.Tensor
    interleaved: bool = False
    positions: Optional[torch.Tensor] = None


def _fit(bits, **numbers):
    """Refuses numbers that a field of so many bits would hold cut (ctypes does so silently)."""
    for what, x in numbers.items():
        if not -(1 << bits - 1) <= x < 1 << bits - 1:
            raise ValueError(f"{what} = {x}: does not fit {bits} bits")


def _ints(t, shape, device, what):
    if t.dtype != torch.int32:
        raise TypeError(f"{what}: {t.dtype} tensor, expected int32")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, the cache is on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {shape}")
    return t.data_ptr()


def _held(name):
    """An attribute whose tensor the library knows by its address: changed in place, never replaced."""
    key = "_" + name

    def get(self):
        return getattr(self, key)

    def put(self, t):
        if self.__dict__.setdefault(key, t) is not t:
            raise ValueError(f"{name}: the calls know this tensor by its address; change it in place "
                             "(+=, copy_), or make a new object around another one")

    return property(get, put)


def _empty_on(device, stream, shape, dtype):
    """Memory that belongs to the work queued on `stream` (None: the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        raise ValueError("a raw stream handle needs explicit outputs and workspace")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace_on(device, stream, nbytes, workspace):
    """The caller's workspace, or one from torch's allocator (None: no bytes), and its size.  The tensor has
    to be held until the call is queued: from then on the stream's order keeps its memory."""
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace: must be contiguous and on {device}")
        return workspace, workspace.numel() * workspace.element_size()
    if nbytes == 0:
        return None, 0
    return _empty_on(device, stream, nbytes, torch.uint8), nbytes


def _queue(call, device, stream, *args):
    """The library's call on `stream` (a stream, its handle, or None: the current one)."""
    index = device.index
    if stream is None:  # (the public current_stream() costs as much as the rest of a call)
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        if stream.device != device:
            raise ValueError(f"stream on {stream.device}, the tensors are on {device}")
        stream = stream.cuda_stream
    if torch.cuda.current_device() == index:
        st = call(*args, stream)
    else:
        with torch.cuda.device(index):
            st = call(*args, stream)
    if st != CFZ_OK:
        raise CfzError(st, call.__name__)


def _rotation(rotation, tokens, device):
    if rotation is None:
        return None
    cos, sin, pos = rotation.cos, rotation.sin, rotation.positions
    if cos.dim() != 2 or cos.shape != sin.shape:
        raise ValueError("rotation: cos and sin must be [rows, rot_dim / 2]")
    for t in (cos, sin):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.device != device:
            raise ValueError("rotation: cos and sin must be contiguous fp32 tensors on "
                             "the cache's device")
    return C.byref(cfz_kv8_rotation(
        cos.data_ptr(), sin.data_ptr(),
        None if pos is None else _ints(pos, (tokens,), device, "positions"),
        cos.shape[0], 2 * cos.shape[1], bool(rotation.interleaved)))


def _rows(t, heads, dim, device, what):
    """[tokens, heads, dim] with dense rows; returns the row stride in elements."""
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, the cache is on {device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{what}: shape {tuple(shape)}, expected [tokens, {heads}, {dim}]")
    if (stride[2] != 1 or (heads > 1 and stride[1] != dim)) and t.numel():
        raise ValueError(f"{what}: a token's heads must lie side by side (strides {stride})")
    return stride[0] if shape[0] > 1 else heads * dim


class Cache:
    """A pool of ``pages`` pages of ``page_tokens`` tokens for ``kv_heads`` heads of ``head_dim``.

    k [pages, kv_heads, page_tokens, head_dim] and v [pages, kv_heads, head_dim, page_tokens]
    hold the codes (int8, or float8_e4m3fn for ``fmt="e4m3"``), k_scale and v_scale [pages,
    kv_heads] their fp32 scales, k_mean [pages, kv_heads, head_dim] the pages' mean keys
    (``pooled=True``; needed by ``select``).

    Every call describes a ragged batch: ``page_table`` [batch, width] int32 with the sequences'
    pages, ``lengths`` [batch] int32, ``offsets`` [batch + 1] int32 with the token rows of each
    sequence, and an upper bound of one sequence's rows known on the host.  Work is queued on
    ``stream`` (default: the current one of the cache's device); with another stream than the
    current one the caller orders the tensors' other uses, as for every call of the library.
    Nothing is recorded for autograd: results carry no gradient, whatever the inputs require.

    The calls know the cache's tensors by their addresses: they may be changed in place, and another tensor
    in their place is refused (ValueError; ``Cache.over`` makes a cache around other ones).

    int8 is the finer of the two where a head's channels are of one size.  Channels many times
    larger than the others leave the others only a few of its steps: e4m3 is meant for such tensors."""

    k, v, k_scale, v_scale, k_mean = map(_held, ("k", "v", "k_scale", "v_scale", "k_mean"))

    def __init__(self, pages, kv_heads, head_dim, page_tokens=64, fmt="int8", pooled=True,
                 device="cuda"):
        if fmt not in FORMATS:
            raise ValueError(f"fmt = {fmt!r}: 'int8' or 'e4m3'")
        code = torch.int8 if fmt == "int8" else torch.float8_e4m3fn

        def zeros(dtype, *shape):
            return torch.zeros(shape, dtype=dtype, device=device)

        self._hold(zeros(torch.uint8, pages, kv_heads, page_tokens, head_dim).view(code),
                   zeros(torch.uint8, pages, kv_heads, head_dim, page_tokens).view(code),
                   zeros(torch.float32, pages, kv_heads), zeros(torch.float32, pages, kv_heads),
                   zeros(torch.float32, pages, kv_heads, head_dim) if pooled else None)

    @classmethod
    def over(cls, k, v, k_scale, v_scale, k_mean=None):
        """A cache around buffers that already hold one (checkpoint and resume)."""
        self = cls.__new__(cls)
        self._hold(k, v, k_scale, v_scale, k_mean)
        return self

    def _hold(self, k, v, k_scale, v_scale, k_mean):
        if k.dim() != 4 or k.dtype not in _CODES:
            raise TypeError("k: expected int8 or float8_e4m3fn [pages, heads, tokens, dim]")
        pages, heads, tokens, dim = k.shape
        for t, shape, dtype, what in (
                (v, (pages, heads, dim, tokens), k.dtype, "v"),
                (k_scale, (pages, heads), torch.float32, "k_scale"),
                (v_scale, (pages, heads), torch.float32, "v_scale"),
                (k_mean, (pages, heads, dim), torch.float32, "k_mean")):
            if t is None and what == "k_mean":
                continue
            if tuple(t.shape) != shape or t.dtype != dtype:
                raise ValueError(f"{what}: {t.dtype} {tuple(t.shape)}, expected {dtype} {shape}")
        held = [t for t in (k, v, k_scale, v_scale, k_mean) if t is not None]
        if any(t.device != k.device for t in held) or not k.is_cuda:
            raise ValueError("the cache's tensors must be on one GPU")
        if not all(t.is_contiguous() for t in held):
            raise ValueError("the cache's tensors must be contiguous")
        self.k, self.v, self.k_scale, self.v_scale, self.k_mean = k, v, k_scale, v_scale, k_mean
        self.pages, self.kv_heads, self.page_tokens, self.head_dim = pages, heads, tokens, dim
        self.device = k.device
        self.desc = cfz_kv8_cache(pages, heads, dim, tokens, _CODES[k.dtype], k.data_ptr(),
                                  v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                  None if k_mean is None else k_mean.data_ptr())
        self._ref = C.byref(self.desc)

    # ---- marshalling

    def _batch(self, page_table, lengths, offsets, tokens, max_rows):
        if page_table.dim() != 2:
            raise ValueError("page_table: expected [batch, width]")
        batch, width = page_table.shape
        if not (batch < 1 << 31 and width < 1 << 31 and -(1 << 63) <= max_rows < 1 << 63):
            _fit(32, batch=batch, table_width=width)
            _fit(64, max_rows=max_rows)
        return cfz_kv8_batch(batch, width, _ints(page_table, None, self.device, "page_table"),
                             _ints(offsets, (batch + 1,), self.device, "offsets"),
                             _ints(lengths, (batch,), self.device, "lengths"), tokens, max_rows)

    def _empty(self, stream, shape, dtype):
        return _empty_on(self.device, stream, shape, dtype)

    def _fill(self, t, value, stream):
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, self.device)
        if stream is None:
            t.fill_(value)
        else:
            with torch.cuda.stream(stream):
                t.fill_(value)

    def _call(self, call, stream, *args):
        index = self.device.index
        if stream is None:  # (the public current_stream() costs as much as the rest of a call)
            stream = torch._C._cuda_getCurrentRawStream(index)
        elif not isinstance(stream, int):
            if stream.device != self.device:
                raise ValueError(f"stream on {stream.device}, the cache is on {self.device}")
            stream = stream.cuda_stream
        if torch.cuda.current_device() == index:
            st = call(*args, stream)
        else:
            with torch.cuda.device(index):
                st = call(*args, stream)
        if st != CFZ_OK:
            raise CfzError(st, call.__name__)

    def _new_rows(self, k, v):
        """Row strides of new keys and values."""
        ks = _rows(k, self.kv_heads, self.head_dim, self.device, "k")
        vs = _rows(v, self.kv_heads, self.head_dim, self.device, "v")
        if k.dtype not in _REALS or v.dtype != k.dtype:
            raise TypeError(f"k and v: {k.dtype} and {v.dtype}, expected one of bf16, fp16, fp32")
        if k.shape[0] != v.shape[0]:
            raise ValueError(f"k has {k.shape[0]} token rows, v {v.shape[0]}")
        return ks, vs

    def _turn(self, rotation, tokens):
        return _rotation(rotation, tokens, self.device)

    def _outputs(self, q, out):
        """Row stride of given outputs."""
        stride = _rows(out, q.shape[1], self.head_dim, self.device, "out")
        if out.dtype != q.dtype or out.shape != q.shape:
            raise ValueError("out: must have q's shape and dtype")
        return stride

    def _fits(self, call, batch, *args):
        """Raises what the library refuses about a call whose tensors (of token rows, queries,
        lists) are left out of ``args``: they are the last thing that it asks for before a workspace."""
        status = call(self._ref, C.byref(batch), *args)
        if status != CFZ_ERR_NULL:
            raise CfzError(status, call.__name__)

    # ---- calls

    def append(self, k, v, page_table, lengths, offsets, max_new, rotation=None, stream=None):
        """Appends token rows k, v [tokens, kv_heads, head_dim] (bf16, fp16 or fp32; the rows may
        be strided) behind the ``lengths`` tokens each sequence holds, the keys rotated on the way.
        The caller adds the new counts to its lengths."""
        ks, vs = self._new_rows(k, v)
        rot = self._turn(rotation, k.shape[0])
        batch = self._batch(page_table, lengths, offsets, k.shape[0], max_new)
        self._call(_lib.cfz_kv8_append, stream, self._ref, C.byref(batch), _REALS[k.dtype],
                   k.data_ptr(), v.data_ptr(), ks, vs, rot)

    def gather(self, page_table, start, offsets, tokens, max_count, dtype=torch.bfloat16, k=None,
               v=None, stream=None):
        """Token rows (k, v) [tokens, kv_heads, head_dim] as numbers: row offsets[b] + i is token
        start[b] + i of sequence b.  k and v may be given; else both are allocated (rows of
        no sequence are then left unset)."""
        shape = (tokens, self.kv_heads, self.head_dim)
        if k is None and v is None:
            k = self._empty(stream, shape, dtype)
            v = self._empty(stream, shape, dtype)
        for t, what in ((k, "k"), (v, "v")):
            if t is not None and (tuple(t.shape) != shape or t.dtype != dtype or
                                  t.device != self.device or not t.is_contiguous()):
                raise ValueError(f"{what}: expected a contiguous {dtype} tensor {shape}")
        if dtype not in _REALS:
            raise TypeError(f"dtype = {dtype}: expected bf16, fp16 or fp32")
        batch = self._batch(page_table, start, offsets, tokens, max_count)
        self._call(_lib.cfz_kv8_gather, stream, self._ref, C.byref(batch), _REALS[dtype],
                   None if k is None else k.data_ptr(), None if v is None else v.data_ptr())
        return k, v

    def _queries(self, q):
        if q.dim() != 3 or q.shape[1] % self.kv_heads or q.shape[1] == 0:
            raise ValueError(f"q: shape {tuple(q.shape)}, expected [tokens, a multiple of "
                             f"{self.kv_heads}, {self.head_dim}]")
        if q.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"q: {q.dtype}, expected bf16 or fp16")
        return _rows(q, q.shape[1], self.head_dim, self.device, "q")

    def _lists(self, blocks, batch, max_q, q_block, count=None):
        _fit(32, q_block=q_block)
        shape = (batch.batch, -(-max_q // q_block), self.kv_heads,
                 count if count is not None else blocks.shape[-1])
        return cfz_kv8_blocks(_ints(blocks, shape, self.device, "blocks"), shape[-1], q_block)

    def attend(self, q, page_table, lengths, offsets, max_q, max_kv, causal=False, scale=None,
               blocks=None, q_block=1, out=None, lse=None, workspace=None, stream=None):
        """Attention of query rows q [tokens, q_heads, head_dim] (bf16 or fp16) over the cache:
        (out, lse), out like q and lse [tokens, q_heads] fp32.  ``scale`` defaults to
        head_dim ** -0.5.  ``blocks`` [batch, ceil(max_q / q_block), kv_heads, count] (from
        ``select``) restricts each block of q_block queries to its listed pages.  Outputs that are
        not given are allocated (rows of no sequence are then left unset)."""
        stride = self._queries(q)
        tokens, heads = q.shape[:2]
        _fit(64, max_kv=max_kv)
        batch = self._batch(page_table, lengths, offsets, tokens, max_q)
        lists = None
        if blocks is not None:
            if q_block < 1 or blocks.dim() != 4:
                raise ValueError("blocks: expected [batch, query blocks, kv_heads, count] and "
                                 "q_block >= 1")
            lists = C.byref(self._lists(blocks, batch, max_q, q_block))
        need = _lib.cfz_kv8_attend_workspace_bytes(self._ref, C.byref(batch), heads,
                                                   max_kv, lists)
        workspace, have = _workspace_on(self.device, stream, need, workspace)
        ostride = heads * self.head_dim
        if out is None:
            out = self._empty(stream, (tokens, heads, self.head_dim), q.dtype)
        else:
            ostride = self._outputs(q, out)
        if lse is None:
            lse = self._empty(stream, (tokens, heads), torch.float32)
        elif (lse.shape != (tokens, heads) or lse.dtype != torch.float32 or
              lse.device != self.device or not lse.is_contiguous()):
            raise ValueError(f"lse: expected a contiguous fp32 tensor {(tokens, heads)}")
        self._call(_lib.cfz_kv8_attend, stream, self._ref, C.byref(batch), _REALS[q.dtype],
                   q.data_ptr(), stride, heads, bool(causal),
                   self.head_dim ** -0.5 if scale is None else scale, max_kv, lists,
                   out.data_ptr(), ostride, lse.data_ptr(),
                   None if workspace is None else workspace.data_ptr(), have)
        return out, lse

    def select(self, q, page_table, lengths, offsets, max_q, max_kv, q_block, count, first=0,
               last=0, causal=False, blocks=None, workspace=None, stream=None):
        """For each block of ``q_block`` queries and each KV head the ``count`` pages whose mean
        keys have the largest product with the block's summed queries, the ``first`` and ``last``
        visible pages always among them: int32 [batch, ceil(max_q / q_block), kv_heads, count],
        ascending page indices of the sequence, padded with -1."""
        stride = self._queries(q)
        if self.k_mean is None:
            raise ValueError("select needs a cache with k_mean (pooled=True)")
        if q_block < 1 or count < 1:
            raise ValueError(f"q_block = {q_block}, count = {count}: at least 1")
        _fit(32, q_block=q_block, count=count, first=first, last=last)
        _fit(64, max_kv=max_kv)
        batch = self._batch(page_table, lengths, offsets, q.shape[0], max_q)
        if blocks is None:
            blocks = self._empty(stream, (batch.batch, -(-max_q // q_block), self.kv_heads, count),
                                 torch.int32)
        lists = self._lists(blocks, batch, max_q, q_block, count)
        need = _lib.cfz_kv8_select_workspace_bytes(self._ref, C.byref(batch), max_kv,
                                                   C.byref(lists))
        workspace, have = _workspace_on(self.device, stream, need, workspace)
        self._call(_lib.cfz_kv8_select, stream, self._ref, C.byref(batch), _REALS[q.dtype],
                   q.data_ptr(), stride, q.shape[1], bool(causal), max_kv, first, last,
                   C.byref(lists), None if workspace is None else workspace.data_ptr(), have)
        if q.shape[0] == 0:  # (the library checks such a call and leaves the lists alone)
            self._fill(blocks, -1, stream)
        return blocks

    def copy(self, moves, origin=None, stream=None):
        """Copies whole pages: page moves.source[i] of ``origin`` (another cache with pages of the same
        kind; default: this one) to page moves.target[i], for the first moves.count[0] pairs, or
        all.  Pairs that name a page outside its pool (-1) are left out.  No target may be another
        pair's target or, within one cache, its source."""
        source, target, count = moves.source, moves.target, moves.count
        shape = (source.numel(),)
        if origin is not None and origin.device != self.device:
            raise ValueError(f"origin: on {origin.device}, the cache is on {self.device}")
        self._call(_lib.cfz_kv8_copy, stream, self._ref, None if origin is None else origin._ref,
                   shape[0], _ints(source, shape, self.device, "source"),
                   _ints(target, shape, self.device, "target"),
                   None if count is None else _ints(count, (1,), self.device, "count"))


@dataclass
class Moves:
    """Pages to be copied (``Cache.copy``): ``source`` and ``target`` int32, -1 where there is nothing
    to do; ``count`` int32 [1], how many of them are meant (None: all).  ``left_out`` int32 [batch] (of
    ``Pages.reserve``): how many of a row's new tokens have no place."""

    source: torch.Tensor
    target: torch.Tensor
    count: Optional[torch.Tensor] = None
    left_out: Optional[torch.Tensor] = None


class Pages:
    """Who holds which page of a pool: ``table`` [batch, width] int32 (-1: no page), ``lengths``
    [batch] int32 and ``refs`` [pages] int32, how many places of the table name each page (0: free).
    The tensors are changed in place; ``table`` and ``lengths`` are what the calls of ``Cache`` take.
    Layers whose caches have the same number of pages share one ``Pages``: the moves that a
    call returns are then made in each layer's cache.

        moves, missing = pages.reserve(counts, max_new)  # pages for counts[b] more tokens a row
        cache.copy(moves)                                # shared pages about to be written
        cache.append(k, v, pages.table, pages.lengths, offsets, max_new)
        pages.lengths += counts - moves.left_out         # (rows that are full take no more)

    Every call is queued like those of ``Cache``; nothing is read by the host.  The calls know the three
    tensors by their addresses: another tensor in their place is refused (ValueError)."""

    table, lengths, refs = map(_held, ("table", "lengths", "refs"))

    def __init__(self, table, lengths, refs, page_tokens):
        if not table.is_cuda:
            raise ValueError("table: libcfz takes device tensors")
        if table.dim() != 2 or refs.dim() != 1:
            raise ValueError(f"table {tuple(table.shape)}, refs {tuple(refs.shape)}: expected "
                             "[batch, width] and [pages]")
        self.device = table.device
        batch, width = table.shape
        _fit(32, batch=batch, width=width, page_tokens=page_tokens)
        self.table, self.lengths, self.refs, self.page_tokens = table, lengths, refs, page_tokens
        self.desc = cfz_kv8_pages(refs.numel(), batch, width, page_tokens,
                                  _ints(table, None, self.device, "table"),
                                  _ints(lengths, (batch,), self.device, "lengths"),
                                  _ints(refs, None, self.device, "refs"))
        self._ref = C.byref(self.desc)

    @classmethod
    def empty(cls, pages, batch, width, page_tokens=64, device="cuda"):
        """``batch`` rows of up to ``width`` pages that hold nothing yet."""
        return cls(torch.full((batch, width), -1, dtype=torch.int32, device=device),
                   torch.zeros(batch, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device), page_tokens)

    def _list(self, t, what, like=None):
        if t.dim() != 1 or (like is not None and t.shape != like.shape):
            raise ValueError(f"{what}: shape {tuple(t.shape)}, expected "
                             f"{'[count]' if like is None else tuple(like.shape)}")
        return _ints(t, None, self.device, what)

    def free(self, rows, keep=None, stream=None):
        """Cuts the rows (int32) off behind their first ``keep[i]`` tokens (None: 0); pages that no row
        holds any more are free."""
        _fit(32, rows=rows.numel())
        _queue(_lib.cfz_kv8_free, self.device, stream, self._ref, rows.numel(),
               self._list(rows, "rows"), None if keep is None else self._list(keep, "keep", rows))

    def fork(self, parents, children, stream=None):
        """Row children[i] holds the pages and length of row parents[i] too, instead of its own.
        Nothing is copied until one of them is about to write (``reserve``).  A pair is left out if a
        row is outside the table, if both are one, if an earlier pair has its child, or if
        its child is the parent of any pair."""
        _fit(32, children=children.numel())
        _queue(_lib.cfz_kv8_fork, self.device, stream, self._ref, children.numel(),
               self._list(parents, "parents", children), self._list(children, "children"))

    def reserve(self, counts, max_new, workspace=None, stream=None):
        """Pages for counts[b] (int32 [batch], at most ``max_new``) more tokens behind each row's
        length, and pages of its own where it would write into one that other rows hold too:
        (moves, missing).  ``moves`` [batch] are to be copied in every cache before the tokens are appended.
        ``missing`` (int32 [1]) is 0, or how many more free pages it takes: then nothing has changed.
        ``moves.left_out`` [batch] says how many of a row's counts[b] tokens have no place: those past ``max_new``
        or past the table's end, which ``Cache.append`` drops."""
        _fit(64, max_new=max_new)
        batch = self.table.shape[0]
        counts = _ints(counts, (batch,), self.device, "counts")
        need = _lib.cfz_kv8_reserve_workspace_bytes(self._ref, max_new)
        out = _empty_on(self.device, stream, 3 * batch + 1, torch.int32)
        source, target, left_out, missing = out.split([batch, batch, batch, 1])
        workspace, have = _workspace_on(self.device, stream, need, workspace)
        _queue(_lib.cfz_kv8_reserve_rows, self.device, stream, self._ref, counts, max_new,
               source.data_ptr(), target.data_ptr(), missing.data_ptr(), left_out.data_ptr(),
               None if workspace is None else workspace.data_ptr(), have)
        return Moves(source, target, left_out=left_out), missing

    def compact(self, workspace=None, stream=None):
        """Moves the pages in use to the front of the pool, the highest to the lowest free one:
        (moves, live), the moves to be made in every cache and the number (int32 [1]) of pages in use,
        which are then 0 .. live - 1."""
        most = self.refs.numel() // 2
        need = _lib.cfz_kv8_compact_workspace_bytes(self._ref)
        source, target, live, count = (_empty_on(self.device, stream, n, torch.int32)
                                       for n in (most, most, 1, 1))
        workspace, have = _workspace_on(self.device, stream, need, workspace)
        _queue(_lib.cfz_kv8_compact, self.device, stream, self._ref, source.data_ptr(),
               target.data_ptr(), live.data_ptr(), count.data_ptr(),
               None if workspace is None else workspace.data_ptr(), have)
        return Moves(source, target, count), live
