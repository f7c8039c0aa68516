"""GPU parity of the 8-bit paged K/V cache against its 64-bit model (oracle/kv8.py).

- append: codes, scales and untouched memory bit for bit; mean keys to one fp32 rounding.
- gather: the rounded product of scale and code, bit for bit.
- select: the lists, equal.
- attend: within the bound below, row by row.

Bound of attend, per output element: the weights enter the second product rounded to fp16, half a
step 2^-11 each, so |error| <= 2^-11 sum w|v| from them; a score is an fp32 sum of D exact
products and a few roundings of its factors, off by at most e = (D + 8) 2^-24 max_t sum|q k| + 2^-21
|y| (y, the score as a power of two with the value scale's logarithm, is below 2^8 here), which moves
numerator and denominator by e sum w|v| each; the sums over n keys add 2 n 2^-24 sum w|v|; weights
that fp16 holds as subnormal numbers lose at most 2^-31 of the largest each (2^-25 at a lift of
2^6), n 2^-31 qmax max(scale) in all; the result is rounded once, half a step of |out|.  lse is off by e
plus the fp32 roundings of the sum and the logarithm, n 2^-24 + 2^-21 max(1, |lse|)."""
import sys

import numpy as np
import pytest
import torch

from oracle import kv8 as model

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_activation_residual_amd import cfz, kv8
DEV = "cuda:0"
REAL = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def cumulative(n):
    return ints(np.concatenate([[0], np.cumsum(n)]))


def to64(t):
    return t.detach().cpu().double().numpy()


class Both:
    """A pool on the GPU and its model, pages handed out in shuffled order."""

    def __init__(self, batch, width, heads, dim, page, fmt, seed=0, spare=2, fill=0x5A):
        self.rng = np.random.default_rng(seed)
        pages = batch * width + spare
        self.cache = kv8.Cache(pages, heads, dim, page, fmt, device=DEV)
        self.cache.k.view(torch.uint8).fill_(fill)
        self.cache.v.view(torch.uint8).fill_(fill)
        for t in (self.cache.k_scale, self.cache.v_scale, self.cache.k_mean):
            t.fill_(7.0)
        self.model = model.Pool(pages, heads, dim, page, fmt)
        self.model.ks[:], self.model.vs[:], self.model.km[:] = 7.0, 7.0, 7.0
        self.table = self.rng.permutation(pages)[:batch * width].reshape(batch, width)
        self.heads, self.dim, self.page, self.fmt, self.fill = heads, dim, page, fmt, fill
        self.held = [0] * batch
        self.gen = torch.Generator().manual_seed(seed)

    def rows(self, n, heads=None, dtype=torch.bfloat16, size=1.0):
        x = torch.randn((n, heads or self.heads, self.dim), generator=self.gen) * size
        return x.to(dtype).to(DEV)

    def append(self, counts, k, v, rotation=None, held=None, **kw):
        held = self.held if held is None else held
        self.cache.append(k, v, ints(self.table), ints(held), cumulative(counts),
                          max(counts, default=0), rotation=rotation, **kw)
        at, rot = 0, None
        if rotation is not None:
            rot = (to64(rotation.cos), to64(rotation.sin), rotation.interleaved)
        for b, n in enumerate(counts):
            pos = None
            if rotation is not None and rotation.positions is not None:
                pos = rotation.positions[at:at + n].tolist()
            self.model.append(to64(k[at:at + n]), to64(v[at:at + n]), self.table[b], held[b], rot,
                              pos)
            at += n
        self.held = [h + n for h, n in zip(held, counts)]

    def fill_up(self, lengths, dtype=torch.bfloat16, size=1.0):
        n = sum(lengths)
        self.append(lengths, self.rows(n, dtype=dtype, size=size), self.rows(n, dtype=dtype, size=size))

    def check(self):
        """Codes, scales and means of every live token; everything else as it was."""
        torch.cuda.synchronize()
        m, c = self.model, self.cache
        assert np.array_equal(c.k_scale.cpu().numpy(), m.ks)
        assert np.array_equal(c.v_scale.cpu().numpy(), m.vs)
        km = c.k_mean.cpu().numpy()
        assert np.all(np.abs(km - m.km) <= 2.0 ** -23 * np.abs(m.km) + 1e-44)
        gk = c.k.view(torch.uint8).cpu().numpy()
        gv = c.v.view(torch.uint8).cpu().numpy().transpose(0, 1, 3, 2)
        live = np.zeros((m.pages, self.page), bool)
        for b, n in enumerate(self.held):
            for t in range(min(n, self.table.shape[1] * self.page)):
                p = m.page_of(self.table[b], t // self.page)
                if p is not None:
                    live[p, t % self.page] = True
        sel = np.broadcast_to(live[:, None, :, None], gk.shape)
        for got, want in ((gk, m.k), (gv, m.v)):
            assert np.array_equal(got[sel], model.code_bytes(want, self.fmt)[sel])
            assert (got[~sel] == self.fill).all(), "bytes outside the live tokens changed"


def rotation(rows, rot_dim, style, positions=None):
    freq = 100.0 ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return kv8.Rotation(a.cos().float().to(DEV), a.sin().float().to(DEV), style == "pairs",
                        None if positions is None else ints(positions))


# ------------------------------------------------------------------ append and gather

@pytest.mark.parametrize("heads,dim,page,fmt,dtype,style,rot", [
    (1, 64, 32, "int8", "bf16", None, 0),
    (3, 64, 64, "int8", "f32", "pairs", 64),
    (2, 128, 64, "int8", "f16", "halves", 128),
    (2, 128, 128, "e4m3", "bf16", "pairs", 64),
    (1, 128, 32, "e4m3", "f32", "halves", 72),
    (5, 64, 128, "e4m3", "f16", "halves", 8),
    (2, 64, 32, "int8", "bf16", "pairs", 24),
])
def test_append_in_several_calls(heads, dim, page, fmt, dtype, style, rot):
    x = Both(4, 5, heads, dim, page, fmt, seed=page + dim)
    turn = rotation(5 * page, rot, style) if style else None
    # nothing, one token, an odd run, more than two pages; then single tokens; then runs that start
    # inside a page with larger values (the older codes are coded again)
    for counts, size in (([0, 1, 37, 2 * page + 3], 1.0), ([1, 1, 1, 1], 0.5),
                         ([page, 33, 0, page - 3], 4.0), ([0, 0, 0, 0], 1.0), ([2, 1, 5, 1], 64.0)):
        n = sum(counts)
        say(f"[gpu] append {counts}")
        x.append(counts, x.rows(n, dtype=REAL[dtype], size=size),
                 x.rows(n, dtype=REAL[dtype], size=size), turn)
        x.check()


def test_append_with_positions_and_strided_rows():
    x = Both(2, 3, 2, 64, 32, "int8", seed=5)
    fused = torch.randn((40, 3, 2, 64), generator=x.gen).bfloat16().to(DEV)
    pos = np.random.default_rng(1).integers(-3, 60, 40)  # some outside the table of 50 rows
    x.append([23, 17], fused[:, 1], fused[:, 2], rotation(50, 32, "pairs", pos))
    x.check()


def test_append_overwrites_a_share_at_a_page_border():
    x = Both(1, 4, 2, 64, 32, "e4m3", seed=6)
    x.fill_up([128])
    k, v = x.rows(64, size=3.0), x.rows(64, size=0.1)
    x.append([64], k, v, held=[32])
    x.held = [128]  # the pages behind the rewritten ones are whole and stay
    x.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_special_values(fmt):
    """NaN, infinities, zeros, subnormal and huge values, and quotients on and beside the borders."""
    x = Both(1, 8, 2, 64, 32, fmt, seed=7)
    k, v = x.rows(256, dtype=torch.float32), x.rows(256, dtype=torch.float32)
    k[3, 0, 5], k[4, 1, 7], k[40, 0, 0], v[9, 0, 1], v[10, 1, 2] = (
        float("nan"), float("inf"), float("-inf"), float("inf"), float("nan"))
    k[64:96] = 0.0
    v[64:96] = 0.0
    v[70, 0, 3] = float("inf")
    k[96:128] *= 1e-40
    v[96:128] *= 3e37
    grid = model.e4m3_values()[:127] if fmt == "e4m3" else np.arange(128.0)
    mid = np.float32((grid[1:] + grid[:-1]) / 2)
    edge = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)), grid])
    edge = np.resize(np.float32(edge), 2048)
    edge[0] = grid[-1]
    # scales 1 and 3: a quotient by 3 of a triple is a tie only if it is exact
    k[128:160, 0] = torch.from_numpy(edge.reshape(32, 64)).to(DEV)
    v[128:160, 1] = -3 * k[128:160, 0]
    k[160:192, 1] = k[128:160, 0] * 0.3
    x.append([256], k, v)
    x.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_ties_whose_product_by_the_inverse_scale_is_off(fmt):
    """x = s (k + 1/2) with s = 49, 107 and the like, where x (1 / s) in 64 bits misses the tie."""
    grid = model.e4m3_values()[:127] if fmt == "e4m3" else np.arange(128.0)
    mid = (grid[1:] + grid[:-1]) / 2
    assert any(49.0 * m * (1.0 / 49.0) != m for m in mid)
    row = np.resize(np.concatenate([[grid[-1]], mid, -mid]), 32 * 64).reshape(32, 64)
    steps = np.array([49.0, 98.0 * 2 ** -7, 103.0, 107.0 * 2 ** 9, 161.0, 187.0 * 2 ** -20])
    rows = np.concatenate([row * s for s in steps])[:, None]
    assert np.array_equal(np.float32(rows), rows)
    x = Both(1, 6, 1, 64, 32, fmt, seed=9)
    k = torch.from_numpy(np.float32(rows)).to(DEV)
    x.append([192], k, -k)
    assert np.array_equal(x.model.ks[x.table[0], 0], steps)
    x.check()


def test_append_leaves_out_bad_pages_and_tokens_past_the_table():
    x = Both(3, 3, 1, 64, 32, "int8", seed=8)
    x.table[0, 1], x.table[1, 0] = -1, x.cache.pages
    x.fill_up([90, 40, 130])
    x.held[2] = 96
    x.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,page,fmt", [(64, 32, "int8"), (128, 64, "e4m3"), (64, 128, "e4m3")])
def test_gather(dtype, dim, page, fmt):
    x = Both(3, 4, 3, dim, page, fmt, seed=9)
    x.table[1, 1] = -5
    x.fill_up([3 * page + 7, 2 * page, 1])
    start, counts = [page - 3, 5, 0], [page + 20, page + 9, 1]
    k, v = x.cache.gather(ints(x.table), ints(start), cumulative(counts), sum(counts), max(counts),
                          dtype=REAL[dtype])
    at = 0
    for b, (lo, n) in enumerate(zip(start, counts)):
        for h in range(x.heads):
            for got, i in ((k, 0), (v, 1)):
                want = x.model.dense(x.table[b], h, lo, lo + n)[i]
                # scale times code is rounded to fp32 and then to the output type
                want = torch.from_numpy(np.float32(want)).to(REAL[dtype])
                assert torch.equal(got[at:at + n, h].cpu(), want)
        at += n


def test_gather_of_one_side_and_past_the_table():
    x = Both(1, 2, 1, 64, 32, "int8", seed=10)
    x.fill_up([64])
    v = torch.full((40, 1, 64), 9.0, device=DEV)
    x.cache.gather(ints(x.table), ints([50]), ints([2, 32]), 40, 40, dtype=torch.float32, v=v)
    want = x.model.dense(x.table[0], 0, 50, 80)[1]
    assert np.array_equal(v[2:32, 0].cpu().numpy(), np.float32(want))
    assert (v[:2] == 9).all() and (v[32:] == 9).all()


# ------------------------------------------------------------------ attention

def bound(x, out, lse, size, reach, n, half, scale):
    d = x.dim
    e = (d + 8) * 2.0 ** -24 * reach + 2.0 ** -21 * 2.0 ** 8
    top = float(np.max(x.model.vs)) * model.QMAX[x.fmt]
    tol = (2.0 ** -11 + 2 * e[..., None] + 2 * n * 2.0 ** -24) * size + n * 2.0 ** -31 * top
    return tol * (1 + half) + half * np.abs(out), e + n * 2.0 ** -24 + 2.0 ** -21 * np.maximum(
        1, np.abs(np.where(np.isfinite(lse), lse, 0)))


def check_attend(x, counts, group, causal, dtype, lengths=None, lists=None, q_block=1, scale=None,
                 size=1.0, call=None, max_kv=None, strided=False, max_q=None):
    lengths = x.held if lengths is None else lengths
    heads, n = x.heads * group, sum(counts)
    max_q = max(counts) if max_q is None else max_q
    pad = 3  # rows behind the last sequence
    q = x.rows(n + pad, heads, REAL[dtype], size)
    out = torch.full_like(q, 5.0)
    if strided:
        wide = torch.full((n + pad, 2 * heads, x.dim), 5.0, dtype=q.dtype, device=DEV)
        wide[:, :heads] = q
        q, out = wide[:, :heads], wide[:, heads:]
    lse = torch.full((n + pad, heads), 5.0, device=DEV)
    table, off, length = ints(x.table), cumulative(counts), ints(lengths)
    room = x.table.shape[1] * x.page
    kw = dict(causal=causal, scale=scale, q_block=q_block, out=out, lse=lse)
    if lists is not None:
        kw["blocks"] = lists
    say(f"[gpu] attend q {counts} over {lengths}, group {group}, causal {causal}, {x.fmt}, "
        f"dim {x.dim}, page {x.page}, lists {None if lists is None else tuple(lists.shape)}")
    x.cache.attend(q, table, length, off, max_q, room if max_kv is None else max_kv, **kw)
    torch.cuda.synchronize()
    assert (out[n:] == 5).all() and (lse[n:] == 5).all()
    half = torch.finfo(REAL[dtype]).eps / 2
    scale = x.dim ** -0.5 if scale is None else scale
    at = 0
    for b, c in enumerate(counts):
        ll = None if lists is None else lists[b].cpu().numpy()
        want, wl, size_, reach = x.model.attend(to64(q[at:at + c]), x.table[b], lengths[b], causal,
                                                scale, ll, q_block)
        got, gl = to64(out[at:at + c]), to64(lse[at:at + c])
        to, tl = bound(x, want, wl, size_, reach, max(lengths[b], 1), half, scale)
        assert np.isfinite(got).all()
        worst = (np.abs(got - want) / np.maximum(to, 1e-300)).max(initial=0)
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(gl), empty) and not got[empty].any()
        worst_l = (np.abs(gl[~empty] - wl[~empty]) / tl[~empty]).max(initial=0)
        say(f"      sequence {b}: {worst:.3f} of the bound, lse {worst_l:.3f}")
        assert worst <= 1 and worst_l <= 1
        at += c
    return out, lse


SHAPES = [
    # heads, group, dim, page, fmt, dtype
    (1, 1, 64, 32, "int8", "bf16"),
    (2, 4, 128, 64, "int8", "bf16"),
    (2, 3, 64, 128, "e4m3", "f16"),
    (1, 20, 128, 32, "e4m3", "bf16"),
    (2, 1, 128, 128, "int8", "f16"),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_attend_single_queries(shape, causal):
    heads, group, dim, page, fmt, dtype = shape
    x = Both(5, 8, heads, dim, page, fmt, seed=11)
    x.fill_up([0, 1, page, 3 * page + 17, 7 * page + 31])
    check_attend(x, [1, 1, 1, 1, 1], group, causal, dtype)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_attend_ragged_prompts(shape, causal):
    heads, group, dim, page, fmt, dtype = shape
    x = Both(4, 6, heads, dim, page, fmt, seed=12)
    x.fill_up([5, 4 * page + 5, 0, 2 * page])
    # more queries than keys (causal: the first rows see nothing), no keys at all, no queries
    check_attend(x, [19, 70, 6, 0], group, causal, dtype)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n", [31, 32, 33, 127, 128, 129, 200])
def test_attend_tile_edges(n, causal):
    x = Both(2, 5, 1, 64, 64, "int8", seed=n)
    x.fill_up([n, 320])
    check_attend(x, [n, n], 1, causal, "bf16")


@pytest.mark.parametrize("dim,fmt", [(64, "int8"), (128, "e4m3")])
def test_attend_splits(dim, fmt):
    """A long cache and few rows: the keys are split over work-groups and joined."""
    x = Both(2, 40, 1, dim, 128, fmt, seed=13)
    x.fill_up([40 * 128 - 5, 77])
    check_attend(x, [1, 1], 2, False, "bf16")
    check_attend(x, [70, 3], 1, True, "f16")


@pytest.mark.parametrize("rows", [1, 40, 100])
def test_attend_ignores_memory_behind_the_tokens(rows):
    """e4m3 pages whose unwritten bytes are NaN codes, scales and table entries that nothing may read."""
    x = Both(2, 5, 1, 64, 32, "e4m3", seed=14, fill=0x7F)
    x.fill_up([70, 33])
    x.table[0, 3:], x.table[1, 2:] = -1, 1 << 30
    x.cache.k_scale[x.cache.k_scale == 7.0] = float("nan")
    x.cache.v_scale[x.cache.v_scale == 7.0] = float("nan")
    check_attend(x, [rows, rows], 1, False, "bf16")
    check_attend(x, [rows, rows], 1, True, "bf16", lengths=[65, 1])


@pytest.mark.parametrize("rows", [1, 40, 100])
def test_attend_bad_pages_hold_nothing(rows):
    x = Both(2, 4, 2, 64, 32, "int8", seed=15)
    x.fill_up([100, 128])
    x.table[0, 0], x.table[1, 1], x.table[1, 2] = -1, x.cache.pages, -7
    check_attend(x, [rows, rows], 2, True, "bf16")
    x.table[:] = -1
    check_attend(x, [rows, rows], 2, False, "bf16")


@pytest.mark.parametrize("rows", [1, 40, 100])
def test_attend_sharp_and_flat_scores(rows):
    for size, scale in ((30.0, 0.5), (1e-3, 1e-3), (200.0, 1e-3)):
        x = Both(1, 6, 1, 64, 32, "int8", seed=16)
        x.fill_up([190], size=2.0)
        check_attend(x, [rows], 1, False, "bf16", scale=scale, size=size)


@pytest.mark.parametrize("rows", [1, 40, 100])
def test_attend_pages_of_very_different_size(rows):
    """Value scales from 0 over 1e-20 to 1e4: the large ones must not drown the weights' sum."""
    x = Both(1, 6, 1, 64, 32, "int8", seed=17)
    k, v = x.rows(190), x.rows(190)
    for i, s in enumerate((0.0, 1e-20, 1.0, 1e4, 0.0, 1e-3)):
        v[32 * i:32 * i + 32] *= s
    x.append([190], k, v)
    check_attend(x, [rows], 1, False, "bf16")
    check_attend(x, [rows], 1, True, "bf16", lengths=[31])


@pytest.mark.parametrize("rows", [1, 40, 100])
def test_attend_nan_and_infinite_queries_stay_in_their_rows(rows):
    x = Both(1, 4, 1, 64, 32, "int8", seed=18)
    x.fill_up([100])
    q = x.rows(2 * rows)
    args = (ints(x.table).repeat(2, 1), ints([100, 100]), cumulative([rows, rows]), rows, 128)
    clean, _ = x.cache.attend(q, *args)
    q[rows, 0, 3] = float("nan")
    got, lse = x.cache.attend(q, *args)
    assert got[rows].isnan().all() and lse[rows].isnan().all()
    keep = [i for i in range(2 * rows) if i != rows]
    assert torch.equal(got[keep], clean[keep])
    q[rows, 0, 3] = float("inf")
    got, _ = x.cache.attend(q, *args)
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dim,rows", [(64, 64), (64, 65), (64, 256), (64, 257), (64, 513), (64, 700),
                                      (128, 128), (128, 129), (128, 257), (128, 300)])
def test_attend_row_tiles(dim, rows, causal):
    """Row counts at and beside the heights of the row tiles, with a few and with many keys."""
    x = Both(2, 6, 1, dim, 128, "int8" if dim == 64 else "e4m3", seed=rows)
    x.fill_up([rows // 2, 765])
    check_attend(x, [rows, rows], 1, causal, "bf16")


@pytest.mark.parametrize("max_q,group", [(1, 64), (2, 64), (1, 32), (1, 33)])
def test_attend_many_query_heads_to_one(max_q, group):
    x = Both(2, 4, 1, 64, 32, "int8", seed=28)
    x.fill_up([128, 77])
    check_attend(x, [max_q, 1], group, True, "bf16")


@pytest.mark.parametrize("dim,max_q,keys", [(64, 1, 8300), (128, 3, 8300), (64, 100, 8300),
                                            (128, 100, 8300), (128, 200, 33000), (64, 300, 33000)])
def test_attend_long_sequences_among_many(dim, max_q, keys):
    """More tiles than are cut into equal runs, and sequences whose pages are looked up in
    several goes; most sequences are empty."""
    page = 128
    x = Both(1, -(-keys // page), 1, dim, page, "int8", seed=29, spare=0)
    x.fill_up([keys])
    others = 1030
    x.table = np.repeat(x.table, others + 2, axis=0)
    few = min(max_q, 5)
    check_attend(x, [0] * others + [few, 1], 1, True, "bf16",
                 lengths=[0] * others + [keys, keys - 77], max_q=max_q)


@pytest.mark.parametrize("group,dim", [(1, 64), (40, 128)])
def test_attend_more_query_blocks_than_runs(group, dim):
    x = Both(2, 4, 1, dim, 32, "int8", seed=30)
    x.fill_up([100, 128])
    lists = ints(np.sort(np.argsort(x.rng.random((2, 520, 1, 4)), axis=-1)[..., :2], axis=-1))
    check_attend(x, [520, 515], group, False, "bf16", lists=lists, q_block=1)


def test_attend_lists_longer_than_the_keys():
    """A list may have far more places than max_kv has pages."""
    x = Both(2, 8, 2, 64, 32, "int8", seed=31)
    x.fill_up([5 * 32, 40])
    lists = torch.full((2, 1, 2, 4096), -1, dtype=torch.int32, device=DEV)
    lists[0, 0, :, 4000:4003] = ints([0, 2, 4])
    lists[1, 0, :, 7], lists[1, 0, :, 4095] = 1, 0
    for rows in (1, 70):
        check_attend(x, [rows, rows], 1, True, "bf16", lists=lists, q_block=rows, max_kv=5 * 32)


@pytest.mark.parametrize("rows", [1, 70])
def test_attend_without_keys_or_pages(rows):
    x = Both(2, 4, 2, 64, 32, "int8", seed=32)
    x.fill_up([100, 60])
    q = x.rows(2 * rows)
    args = (ints(x.table), ints(x.held), cumulative([rows, rows]), rows)
    none = kv8.Cache(0, 2, 64, 32, "int8", device=DEV)
    for cache, max_kv in ((x.cache, 0), (none, 128)):
        out, lse = cache.attend(q, *args, max_kv)
        assert not out.any() and torch.isneginf(lse).all()
        assert (cache.select(q, *args, max_kv, 16, 2) == -1).all()
    k, v = none.gather(ints(x.table), ints([0, 0]), cumulative([5, 6]), 11, 6)
    assert not k.any() and not v.any()
    none.append(x.rows(11), x.rows(11), ints(x.table), ints([0, 0]), cumulative([5, 6]), 6)
    torch.cuda.synchronize()


def test_offsets_out_of_order_or_range_are_clamped():
    """Offsets that fall, or pass the token rows, describe sequences that are short or empty."""
    x = Both(4, 4, 1, 64, 32, "int8", seed=33)
    x.fill_up([100, 60, 128, 30])
    table, held = ints(x.table), ints(x.held)
    q = x.rows(20)
    out, lse = torch.full_like(q, 5.0), torch.full((20, 1), 5.0, device=DEV)
    x.cache.attend(q, table, held, ints([-3, 5, 2, -9, 1 << 30]), 15, 128, out=out, lse=lse)
    # sequence 0 has rows 0 .. 4; 1 and 2 have none; 3 has rows 0 .. 14 (of those up to 20)
    a, al = x.cache.attend(q, table[3:].contiguous(), held[3:].contiguous(), ints([0, 15]), 15, 128)
    assert torch.equal(out[5:15], a[5:15]) and torch.equal(lse[5:15], al[5:15])
    assert (out[15:] == 5).all() and (lse[15:] == 5).all()


def test_attend_strided_rows_and_max_kv():
    x = Both(2, 4, 2, 64, 32, "int8", seed=19)
    x.fill_up([100, 61])
    check_attend(x, [9, 40], 2, True, "bf16", strided=True, max_kv=100)
    check_attend(x, [1, 1], 2, True, "f16", strided=True, max_kv=101)


def test_attend_past_four_gib():
    """Page numbers whose byte offsets pass 2^32."""
    pages = (1 << 32) // (8 * 128 * 128) + 40
    cache = kv8.Cache(pages, 8, 128, 128, "int8", pooled=True, device=DEV)
    table = ints([[pages - 1, 3, pages - 30], [pages - 2, pages - 3, 0]])
    gen = torch.Generator(device=DEV).manual_seed(0)
    k = torch.randn((600, 8, 128), generator=gen, device=DEV).bfloat16()
    v = torch.randn((600, 8, 128), generator=gen, device=DEV).bfloat16()
    cache.append(k, v, table, ints([0, 0]), cumulative([300, 300]), 300)
    gk, gv = cache.gather(table, ints([0, 0]), cumulative([300, 300]), 600, 300,
                          dtype=torch.float32)
    small = kv8.Cache(6, 8, 128, 128, "int8", device=DEV)
    t2 = ints([[0, 1, 2], [3, 4, 5]])
    small.append(k, v, t2, ints([0, 0]), cumulative([300, 300]), 300)
    sk, sv = small.gather(t2, ints([0, 0]), cumulative([300, 300]), 600, 300, dtype=torch.float32)
    assert torch.equal(gk, sk) and torch.equal(gv, sv)
    q = torch.randn((82, 8, 128), generator=gen, device=DEV).bfloat16()
    for counts in ([1, 1], [41, 41]):
        n = sum(counts)
        a = cache.attend(q[:n], table, ints([300, 300]), cumulative(counts), max(counts), 384)
        b = small.attend(q[:n], t2, ints([300, 300]), cumulative(counts), max(counts), 384)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        bl = [c.select(q[:n], t, ints([300, 300]), cumulative(counts), max(counts), 384, 8, 2)
              for c, t in ((cache, table), (small, t2))]
        assert torch.equal(*bl)


# ------------------------------------------------------------------ selection

def check_select(x, counts, group, q_block, count, first, last, causal, lengths=None,
                 dtype="bf16"):
    lengths = x.held if lengths is None else lengths
    q = x.rows(sum(counts), x.heads * group, REAL[dtype])
    room = x.table.shape[1] * x.page
    got = x.cache.select(q, ints(x.table), ints(lengths), cumulative(counts), max(counts), room,
                         q_block, count, first, last, causal).cpu().numpy()
    at = 0
    x.model.km = x.cache.k_mean.cpu().numpy()
    for b, n in enumerate(counts):
        want = x.model.select(to64(q[at:at + n]), x.table[b], lengths[b], causal, q_block, count,
                              first, last)
        assert np.array_equal(got[b, :len(want)], want), f"sequence {b}"
        assert (got[b, len(want):] == -1).all()
        at += n
    return q


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads,group,dim,page,q_block,count,first,last", [
    (2, 1, 64, 32, 1, 3, 0, 0),
    (1, 4, 128, 64, 16, 5, 1, 2),
    (3, 2, 64, 32, 64, 1, 0, 0),
    (1, 1, 128, 32, 7, 4, 2, 2),
    (1, 1, 64, 32, 1000, 40, 1, 1),
])
def test_select(heads, group, dim, page, q_block, count, first, last, causal):
    x = Both(5, 12, heads, dim, page, "int8", seed=20)
    x.fill_up([0, 3, 12 * page, 5 * page + 1, 9 * page - 1])
    x.table[2, 4], x.table[2, 7] = -1, x.cache.pages + 3
    check_select(x, [2, 5, 1, 70, 33], group, q_block, count, first, last, causal)


def test_select_ties_go_to_the_lower_page():
    x = Both(1, 600, 1, 64, 32, "int8", seed=21)
    x.held = [600 * 32]
    x.cache.k_mean.copy_(torch.tensor([1.0, -1.0, 0.5], device=DEV)[torch.arange(
        x.cache.pages, device=DEV) % 3][:, None, None].expand_as(x.cache.k_mean))
    for count in (1, 100, 301, 599):
        check_select(x, [4], 1, 2, count, 0, 0, False)
    x.cache.k_mean.fill_(float("nan"))
    x.cache.k_mean[x.table[0, 500]] = -1e30
    check_select(x, [4], 1, 2, 9, 0, 0, False)


@pytest.mark.parametrize("heads,group,q_block,count,counts,causal", [
    (2, 1, 1, 2, [1, 1, 1], False),
    (1, 4, 1, 3, [9, 1, 0], True),
    (2, 1, 64, 3, [70, 129, 1], True),
    (1, 3, 16, 2, [70, 5, 40], False),
    (1, 1, 128, 1, [200, 3, 130], True),
    (2, 2, 33, 5, [100, 34, 2], True),
])
def test_attend_over_selected_pages(heads, group, q_block, count, counts, causal):
    x = Both(3, 7, heads, 64, 32, "int8", seed=22)
    x.fill_up([200, 7 * 32, 5])
    q = check_select(x, counts, group, q_block, count, 0, 1, causal)
    room = 7 * 32
    lists = x.cache.select(q, ints(x.table), ints(x.held), cumulative(counts), max(counts), room,
                           q_block, count, 0, 1, causal)
    check_attend(x, counts, group, causal, "bf16", lists=lists, q_block=q_block)


def test_attend_over_long_lists_and_bad_entries():
    x = Both(1, 64, 1, 128, 64, "e4m3", seed=23)
    x.fill_up([64 * 64 - 9])
    lists = torch.full((1, 1, 1, 48), -1, dtype=torch.int32, device=DEV)
    lists[0, 0, 0, :41] = ints(np.sort(x.rng.permutation(64)[:41]))
    check_attend(x, [1], 4, False, "bf16", lists=lists)
    lists[0, 0, 0, 45], lists[0, 0, 0, 46], lists[0, 0, 0, 47] = 64, 2 ** 31 - 1, -2 ** 31
    check_attend(x, [50], 1, True, "bf16", lists=lists, q_block=50)
    check_attend(x, [1], 1, False, "bf16", lists=torch.full_like(lists, -1))


# ------------------------------------------------------------------ as it is used

def test_codec_to_cache_to_attention():
    """Two shares received through the codec, appended from the fp32 bases, attended over; three
    denoising steps, the shares rewritten at their page borders each step."""
    heads, dim, rows, page = 4, 64, 96, 32
    x = Both(1, 6, heads, dim, page, "int8", seed=24)
    cols = heads * dim
    x0 = [torch.randn((rows, cols), generator=x.gen).bfloat16().to(DEV) for _ in range(4)]
    snd = [cfz.Sender(rows, cols, x0=t) for t in x0]
    rcv = [cfz.Receiver(rows, cols, x0=t) for t in x0]
    turn = rotation(2 * rows, dim, "pairs")
    for step in range(3):
        for i in range(4):
            xt = (x0[i].float() + 0.02 * (step + 1) * torch.randn((rows, cols), generator=x.gen)
                  .to(DEV)).bfloat16()
            rcv[i].decompress(*snd[i].compress(xt))
        for share in range(2):
            k, v = (rcv[2 * share + j].base.view(rows, heads, dim) for j in range(2))
            x.append([rows], k, v, turn, held=[share * rows])
        x.check()
        check_attend(x, [rows], 1, False, "bf16")
        q = check_select(x, [rows], 1, 32, 3, 0, 0, False)
        lists = x.cache.select(q, ints(x.table), ints(x.held), cumulative([rows]), rows, 192, 32, 3)
        check_attend(x, [rows], 1, False, "bf16", lists=lists, q_block=32)


@pytest.mark.parametrize("count,group", [(None, 1), (3, 2)])
def test_layers_of_shares_on_streams(count, group):
    """Three layers over an own share and two received ones of other sizes, two items each: on
    two streams eagerly and in a replayed graph, against one stream and the model."""
    from diffusion_activation_residual_amd import cadence
    heads, dim, page, batch, tokens, nq, L = 2, 64, 32, 2, [40, 96, 33], 40, 3
    turn = rotation(sum(tokens), dim, "halves")
    plan = cadence.SharePlan(batch, tokens, nq, page, turn, 16, count, 0, 1, device=DEV)
    gen = torch.Generator().manual_seed(34)

    def randn(n, h):
        return torch.randn((n, h, dim), generator=gen).bfloat16().to(DEV)

    x0 = [[(randn(batch * n, heads), randn(batch * n, heads)) for n in tokens] for _ in range(L)]
    snd = [[[cfz.Sender(len(t), heads * dim, x0=t) for t in pair] for pair in layer[1:]]
           for layer in x0]
    q = [randn(batch * nq, heads * group) for _ in range(L)]

    class Side:
        def __init__(self):
            self.rcv = [[[cfz.Receiver(len(t), heads * dim, x0=t) for t in pair]
                         for pair in layer[1:]] for layer in x0]
            self.own = [[t.clone() for t in layer[0]] for layer in x0]
            self.caches = [kv8.Cache(plan.pages, heads, dim, page, device=DEV) for _ in range(L)]
            self.out = [torch.full_like(t, 5.0) for t in q]

        def step(self, streams):
            layers = [[cadence.Share(*self.own[l])] +
                      [cadence.Share(*(r.base.view(-1, heads, dim) for r in rs),
                                     tuple(r.handle for r in rs), tuple(s.codes for s in ss),
                                     tuple(s.scales for s in ss))
                       for rs, ss in zip(self.rcv[l], snd[l])] for l in range(L)]
            cadence.enqueue_layer_attention(plan, layers, self.caches, q, self.out, streams)

    a, b, g = Side(), Side(), Side()
    cap = torch.cuda.Stream()
    streams = [torch.cuda.current_stream(), torch.cuda.Stream()]
    for step in range(4):
        for l in range(L):
            for side in (a, b, g):
                for t, z in zip(side.own[l], x0[l][0]):
                    t.copy_(z * (1.0 + step))
            for pair, ss in zip(x0[l][1:], snd[l]):
                for t, s in zip(pair, ss):
                    s.compress((t.float() * (1.0 + 0.1 * step)).bfloat16())
        say(f"[gpu] step {step}")
        a.step(streams)
        b.step(streams[:1])
        if step == 0:
            torch.cuda.synchronize()
            g.step(streams[:1])  # (the captured step starts from the second one)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=cap):
                g.step([cap, streams[1]])
        else:
            graph.replay()
        torch.cuda.synchronize()
        for l in range(L):
            for side in (b, g):
                assert torch.equal(a.out[l], side.out[l]), f"step {step}, layer {l}"
                assert torch.equal(a.caches[l].k, side.caches[l].k)
                assert torch.equal(a.caches[l].v, side.caches[l].v)
    x = Both(batch, plan.width, heads, dim, page, "int8", spare=0)
    x.cache, x.table, x.held = a.caches[0], plan.table.cpu().numpy(), [sum(tokens)] * batch
    x.model.ks[:], x.model.vs[:], x.model.km[:] = 0, 0, 0
    x.fill = 0  # (the pool was allocated as zeros)
    rot = (to64(turn.cos), to64(turn.sin), False)
    shares = [a.own[0]] + [[r.base.view(-1, heads, dim) for r in rs] for rs in a.rcv[0]]
    # (every step writes all shares from the first token on: earlier steps leave nothing)
    for item in range(batch):
        for i, n in enumerate(tokens):
            k, v = (to64(t[item * n:(item + 1) * n]) for t in shares[i])
            x.model.append(k, v, x.table[item], sum(tokens[:i]), rot, None)
    x.check()
    check_attend(x, [nq] * batch, group, False, "bf16")
    lists = None
    if count:
        lists = a.caches[0].select(q[0], plan.table, plan.lengths, plan.q_offsets, nq, plan.tokens,
                                   16, count, 0, 1)
    want, _ = a.caches[0].attend(q[0], plan.table, plan.lengths, plan.q_offsets, nq, plan.tokens,
                                 blocks=lists, q_block=16)
    assert torch.equal(a.out[0], want)


@pytest.mark.parametrize("rows", [1, 48])
def test_captured_step_replays_like_eager(rows):
    """Append, select and both attentions in one HIP graph: lengths on the device move on from replay
    to replay, and every replay equals the eager calls on a second cache."""
    def make():
        x = Both(2, 40, 2, 64, 32, "int8", seed=25)
        x.fill_up([500, 300])
        return x

    a, b = make(), make()
    table, off = ints(a.table), cumulative([rows, rows])
    k, v = a.rows(2 * rows), a.rows(2 * rows)
    q = a.rows(2 * rows, 4)
    la, lb = ints(a.held), ints(a.held)

    def step(c, length):
        c.append(k, v, table, length, off, rows)
        length += rows
        out, lse = c.attend(q, table, length, off, rows, 1280, causal=True)
        lists = c.select(q, table, length, off, rows, 1280, 16, 4, 1, 1, causal=True)
        return (out, lse, lists) + c.attend(q, table, length, off, rows, 1280, causal=True,
                                            blocks=lists, q_block=16)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a.cache, la)  # warm-up
    torch.cuda.current_stream().wait_stream(side)
    step(b.cache, lb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(a.cache, la)
    for i in range(4):
        k.copy_(a.rows(2 * rows, size=1.0 + i))
        q.copy_(a.rows(2 * rows, 4))
        graph.replay()
        want = step(b.cache, lb)
        torch.cuda.synchronize()
        assert torch.equal(la, lb)
        for got, w in zip(outs, want):
            assert torch.equal(got, w), f"replay {i}"
        assert torch.equal(a.cache.k, b.cache.k) and torch.equal(a.cache.v, b.cache.v)


def test_calls_on_two_streams_at_once():
    x = Both(2, 40, 2, 64, 32, "int8", seed=26)
    x.fill_up([1200, 900])
    q = x.rows(2, 4)
    args = (ints(x.table), ints(x.held), cumulative([1, 1]), 1, 1280)
    want = x.cache.attend(q, *args)
    wl = x.cache.select(q, *args, 1, 4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s in streams:
            got.append((x.cache.attend(q, *args, stream=s), x.cache.select(q, *args, 1, 4, stream=s)))
    torch.cuda.synchronize()
    for (o, l), bl in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1]) and torch.equal(bl, wl)


def test_binding_refusals():
    x = Both(1, 2, 2, 64, 32, "int8", seed=27)
    c, t, n, off = x.cache, ints(x.table), ints([0]), ints([0, 4])
    k = x.rows(4)
    with pytest.raises(TypeError):
        c.append(k.double(), k.double(), t, n, off, 4)
    with pytest.raises(ValueError):
        c.append(k, k[:3], t, n, off, 4)
    with pytest.raises(ValueError):
        c.append(k[:, :1], k[:, :1], t, n, off, 4)
    with pytest.raises(ValueError):
        c.append(k.cpu(), k.cpu(), t, n, off, 4)
    with pytest.raises(TypeError):
        c.append(k, k, t.long(), n, off, 4)
    with pytest.raises(ValueError):
        c.append(k, k, t, n, ints([0, 1, 4]), 4)
    with pytest.raises(cfz.CfzError):
        c.append(k[:1].expand(4, -1, -1), k, t, n, off, 4)
    with pytest.raises(ValueError):
        c.attend(x.rows(4, 3), t, n, off, 4, 64)
    with pytest.raises(TypeError):
        c.attend(k.float(), t, n, off, 4, 64)
    with pytest.raises(cfz.CfzError):
        c.attend(k, t, n, off, 4, 65)
    with pytest.raises(ValueError):
        c.attend(k, t, n, off, 4, 64, blocks=torch.zeros((1, 2, 2, 3), dtype=torch.int32, device=DEV),
                 q_block=4)
    with pytest.raises(ValueError):
        c.select(k, t, n, off, 4, 64, 0, 1)
    with pytest.raises(cfz.CfzError):
        c.select(k, t, n, off, 4, 64, 1, 2, first=2, last=1)
    with pytest.raises(ValueError):
        kv8.Cache.over(c.k, c.v, c.k_scale, c.v_scale[:1])
    with pytest.raises(TypeError):
        kv8.Cache.over(c.k.view(torch.uint8), c.v, c.k_scale, c.v_scale)
