"""The codec at model cadence: one grouped compress and one grouped decode per layer (its K and
V, which the sender has together once the layer's QKV projection is done), with the layers
spread round-robin over several streams so that one layer's launches overlap another's.

Patch parallelism exchanges each layer's K and V once per denoising step (paper: reproducibility
table, "Pseudocode", Algorithm 1: project QKV, all-gather K and V, attention).  Layer l's codec
work touches only layer l's states and payload buffers, so its compress and decode keep their
order on one stream while other layers' launches run beside them on other streams; each
launch's ramp-up and drain then overlap another launch's streaming.

``enqueue_layer_attention`` goes on to the algorithm's next line: what a device has received of
every share's K and V is decoded, the shares are written into the layer's 8-bit cache, and the
device's own queries attend over all of them.

Host logic only: every launch is a call of the C ABI through the binding."""
import ctypes as C
from contextlib import contextmanager
from dataclasses import dataclass
from typing import Optional

import torch

from . import cfz, kv8


@dataclass
class Share:
    """One device's part of a layer's tokens: ``k`` and ``v`` [batch * tokens, kv_heads, head_dim]
    (bf16, fp16 or fp32), the batch's items one after the other -- the receivers' bases viewed so
    for what comes through the codec, the projections themselves for the device's own part.

    ``receivers`` (state handles), ``codes`` and ``scales``: (K's, V's) of a share that is decoded
    first; None for one that is there already (the own one, or the uncompressed first step)."""

    k: torch.Tensor
    v: torch.Tensor
    receivers: Optional[tuple] = None
    codes: Optional[tuple] = None
    scales: Optional[tuple] = None


class SharePlan:
    """What the layers of one model have in common: ``batch`` items whose tokens are split into
    shares of ``share_tokens`` tokens each, ``queries`` queries an item, the page table (each item has
    its own of the pages 0 .. pages - 1 of a pool), and the rotation of the keys.

    With ``count`` the queries attend in blocks of ``q_block`` over the ``count`` pages that
    ``kv8.Cache.select`` picks for them, the ``first`` and ``last`` ones always among them."""

    def __init__(self, batch, share_tokens, queries, page_tokens, rotation=None, q_block=128,
                 count=None, first=0, last=0, scale=None, device="cuda"):
        share_tokens = list(share_tokens)
        if batch < 1 or not share_tokens or min(share_tokens) < 1 or queries < 1:
            raise ValueError(f"batch = {batch}, share_tokens = {share_tokens}, queries = {queries}: "
                             "at least one of each")
        if page_tokens not in (32, 64, 128):
            raise ValueError(f"page_tokens = {page_tokens}: 32, 64 or 128")
        if count is not None and (not 1 <= count <= 4096 or not 1 <= q_block < 1 << 31 or
                                  first < 0 or last < 0 or first + last > count):
            raise ValueError(f"count = {count}, q_block = {q_block}, first = {first}, last = {last}")
        self.batch, self.share_tokens, self.queries = batch, share_tokens, queries
        self.tokens = sum(share_tokens)
        self.page_tokens = page_tokens
        self.width = -(-self.tokens // page_tokens)
        self.pages = batch * self.width
        self.rotation, self.scale = rotation, scale
        self.q_block, self.count, self.first, self.last = q_block, count, first, last

        def ints(x):
            return torch.tensor(x, dtype=torch.int32, device=device)

        self.table = torch.arange(self.pages, dtype=torch.int32, device=device).view(batch, -1)
        starts = [sum(share_tokens[:i]) for i in range(len(share_tokens))]
        self.starts = [ints([s] * batch) for s in starts]
        self.offsets = [ints([i * n for i in range(batch + 1)]) for n in share_tokens]
        self.lengths = ints([self.tokens] * batch)
        self.q_offsets = ints([i * queries for i in range(batch + 1)])

    def _check_sizes(self, cache, q, keys):
        """Raises what the library refuses about these sizes."""
        for i, k in enumerate(keys):
            batch = cache._batch(self.table, self.starts[i], self.offsets[i], len(k),
                                 self.share_tokens[i])
            row = cache.kv_heads * cache.head_dim
            cache._fits(kv8._lib.cfz_kv8_append, batch, kv8._REALS[k.dtype], None, None, row, row,
                        cache._turn(self.rotation, len(k)), None)
        batch = cache._batch(self.table, self.lengths, self.q_offsets, len(q), self.queries)
        heads, dtype = q.shape[1], kv8._REALS[q.dtype]
        row, lists = heads * cache.head_dim, None
        if self.count is not None:
            lists = C.byref(kv8.cfz_kv8_blocks(None, self.count, self.q_block))
            cache._fits(kv8._lib.cfz_kv8_select, batch, dtype, None, row, heads, 0, self.tokens,
                        self.first, self.last, lists, None, 0, None)
        scale = cache.head_dim ** -0.5 if self.scale is None else self.scale
        cache._fits(kv8._lib.cfz_kv8_attend, batch, dtype, None, row, heads, 0, scale, self.tokens,
                    lists, None, row, None, None, 0, None)

    def write(self, cache, index, share, stream=None):
        """Writes share ``index`` into its place of the items' sequences.  Shares are written in
        order: a page that two of them share ends with the later one's first tokens."""
        cache.append(share.k, share.v, self.table, self.starts[index], self.offsets[index],
                     self.share_tokens[index], rotation=self.rotation, stream=stream)

    def attend(self, cache, q, out=None, lse=None, stream=None):
        """The queries q [batch * queries, q_heads, head_dim] over all shares: (out, lse)."""
        blocks = None
        if self.count is not None:
            blocks = cache.select(q, self.table, self.lengths, self.q_offsets, self.queries,
                                  self.tokens, self.q_block, self.count, self.first, self.last,
                                  stream=stream)
        return cache.attend(q, self.table, self.lengths, self.q_offsets, self.queries, self.tokens,
                            scale=self.scale, blocks=blocks, q_block=self.q_block, out=out,
                            lse=lse, stream=stream)


def enqueue_layer_step(layers, senders, receivers, x, codes, scales, streams, xhat=None):
    """Enqueue one step: for layer l (a list of tensor indices, e.g. [2l, 2l + 1]) one grouped
    compress of x[i] for i in layers[l], then one grouped decode of the codes it wrote, both on
    streams[l % len(streams)].  The other streams first wait for streams[0] and streams[0]
    finally waits for all of them, so the whole step is ordered after work queued before it on
    streams[0] and before work queued after it.  Works eagerly and under torch.cuda.graph
    capture (streams[0] is then the capture stream).

    senders / receivers: cfz handles per tensor; x, codes, scales (and xhat, or None): device
    tensors per tensor index.  The tensors of different layers must not share buffers."""
    with _spread(streams):
        for l, c in enumerate(layers):
            st = streams[l % len(streams)]
            cfz.cfz_compress_group([senders[i] for i in c], [x[i] for i in c],
                                   [codes[i] for i in c], [scales[i] for i in c], stream=st)
            cfz.cfz_decompress_group([receivers[i] for i in c], [codes[i] for i in c],
                                     [scales[i] for i in c],
                                     None if xhat is None else [xhat[i] for i in c], stream=st)


def enqueue_layer_attention(plan, layers, caches, q, out, streams):
    """Enqueue one step of the attention over compressed shares: for layer l one grouped decode
    of the received payloads of layers[l] (a list of ``Share``, in the order of the plan's shares),
    their tokens into caches[l] (``kv8.Cache`` of at least ``plan.pages`` pages), and the
    attention of q[l] over all of them into out[l], on streams[l % len(streams)], ordered as in
    ``enqueue_layer_step``.  Works eagerly and under capture.  The layers must not share
    caches, tensors or receivers.

    A step that does not fit is refused whole, before anything is queued: a decode moves its
    receivers' bases on, so that a step cannot be tried again after half of it."""
    _check_step(plan, layers, caches, q, out, streams)
    with _spread(streams):
        for l, shares in enumerate(layers):
            st = streams[l % len(streams)]
            got = [s for s in shares if s.receivers is not None]
            if got:
                cfz.cfz_decompress_group(*_payload(got), stream=st)
            for i, s in enumerate(shares):
                plan.write(caches[l], i, s, stream=st)
            # (the log-sum-exp is not wanted: its buffer lives as long as the work on st)
            plan.attend(caches[l], q[l], out=out[l], stream=st)


def _payload(shares):
    return ([r for s in shares for r in s.receivers], [c for s in shares for c in s.codes],
            [c for s in shares for c in s.scales])


def _check_step(plan, layers, caches, q, out, streams):
    """Everything that a launch of the step would refuse."""
    if not streams:
        raise ValueError("at least one stream")
    if not len(layers) == len(caches) == len(q) == len(out):
        raise ValueError(f"{len(layers)} layers, {len(caches)} caches, {len(q)} queries and "
                         f"{len(out)} outputs")
    alike = set()  # the plan's sizes are checked once for layers of the same sizes
    for l, (shares, cache) in enumerate(zip(layers, caches)):
        if len(shares) != len(plan.share_tokens):
            raise ValueError(f"layer {l}: {len(shares)} shares, the plan has "
                             f"{len(plan.share_tokens)}")
        for i, s in enumerate(shares):
            if len({s.receivers is None, s.codes is None, s.scales is None}) != 1:
                raise ValueError(f"layer {l}, share {i}: receivers, codes and scales together")
            if s.k.shape[0] != plan.batch * plan.share_tokens[i]:
                raise ValueError(f"layer {l}, share {i}: {s.k.shape[0]} token rows, the plan has "
                                 f"{plan.batch} x {plan.share_tokens[i]}")
        if q[l].shape[0] != plan.batch * plan.queries:
            raise ValueError(f"layer {l}: {q[l].shape[0]} query rows, the plan has "
                             f"{plan.batch} x {plan.queries}")
        if cache.page_tokens != plan.page_tokens or cache.pages < plan.pages:
            raise ValueError(f"layer {l}: a cache of {cache.pages} pages of "
                             f"{cache.page_tokens}, the plan needs {plan.pages} of "
                             f"{plan.page_tokens}")
        if plan.count is not None and cache.k_mean is None:
            raise ValueError(f"layer {l}: selection needs a cache with k_mean (pooled=True)")
        st = streams[l % len(streams)]
        if st.device != cache.device:
            raise ValueError(f"layer {l}: stream on {st.device}, the cache is on {cache.device}")
        for s in shares:
            ks, vs = cache._new_rows(s.k, s.v)
            _whole_rows(s.k, ks, l, "k")
            _whole_rows(s.v, vs, l, "v")
        _whole_rows(q[l], cache._queries(q[l]), l, "q")
        if out[l] is not None:
            _whole_rows(out[l], cache._outputs(q[l], out[l]), l, "out")
        got = [s for s in shares if s.receivers is not None]
        if got:
            cfz.check_decompress_group(*_payload(got))
        sizes = (cache.kv_heads, cache.head_dim, cache.device, q[l].shape[1], q[l].dtype,
                 tuple(s.k.dtype for s in shares))
        if sizes not in alike:
            plan._check_sizes(cache, q[l], [s.k for s in shares])
            alike.add(sizes)


def _whole_rows(t, stride, layer, what):
    """Rows side by side or apart, in 16-byte vectors."""
    _, heads, dim = t.shape
    if (stride < heads * dim or stride >= 1 << 31 or stride * t.element_size() % 16 or
            t.data_ptr() % 16):
        raise ValueError(f"layer {layer}: rows of {what} {stride} elements apart from "
                         f"{t.data_ptr():#x} on, expected at least {heads * dim}, in multiples of "
                         "16 bytes")


@contextmanager
def _spread(streams):
    """streams[1:] start behind what is queued on streams[0], which goes on behind them."""
    if not streams:
        raise ValueError("at least one stream")
    for s in streams[1:]:
        s.wait_stream(streams[0])
    try:
        yield
    finally:
        for s in streams[1:]:
            streams[0].wait_stream(s)
