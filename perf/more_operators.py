"""What lies between a transformer layer's residual stream and the 8-bit K/V cache: what is
measured.

Four groups of operators.  `norm` adds a block's gated output to the residual stream and
normalises the sum for the next block.  `rotate` turns queries and keys by their positions, with
a norm of each head before it, and makes the tables of angles.  `step` and `pack` manage the pages
of a cache: dropped sequences, forked ones, pages for new tokens with copies of the shared ones
that will be written, and a pool packed into its lowest pages.  `adapt` adds the low-rank adapters
of several requests to a projection that they share.
"""
import math

import numpy as np
import torch

own = False

REAL = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases

def _norm(name, batch, rows, cols, real, stream, before, after, modulated, ragged=False):
    return dict(name=name, kind="norm", batch=batch, rows=rows, cols=cols, real=real,
                stream=stream, before=before, after=after, modulated=modulated, ragged=ragged)


def _rotate(name, batch, rows, start, heads, kv_heads, dim, turn, layout, normed, axes, scaling,
            fresh, real, ragged=False):
    return dict(name=name, kind="rotate", batch=batch, rows=rows, start=start, heads=heads,
                kv_heads=kv_heads, dim=dim, turn=turn, layout=layout, normed=normed, axes=axes,
                scaling=scaling, fresh=fresh, real=real, ragged=ragged)


def _step(name, batch, forks, held, new, heads, dim, page):
    return dict(name=name, kind="step", batch=batch, forks=forks, held=held, new=new, heads=heads,
                dim=dim, page=page)


def _pack(name, batch, pages, live, heads, dim, page):
    return dict(name=name, kind="pack", batch=batch, pages=pages, live=live, heads=heads, dim=dim,
                page=page)


def _adapt(name, batch, rows, cols, slices, width, rank, count, real, ragged=False):
    return dict(name=name, kind="adapt", batch=batch, rows=rows, cols=cols, slices=slices,
                width=width, rank=rank, count=count, real=real, ragged=ragged)


def listed():
    return [
        # one token of each of 32 running sequences, root mean square norm with weights: the smallest
        _norm("norm-tokens", 32, 1, 1024, "bf16", "bf16", "rms", "none", False),
        # two items' video shares: gate, scale and shift an item, layer norm without weights
        _norm("norm-video", 2, 4388, 1920, "bf16", "bf16", "layer", "none", True),
        # ragged prompts, a norm on either side of the block, the residual stream in fp32
        _norm("norm-prompts", 7, 2311, 4096, "f16", "f32", "rms", "rms", False, True),
        # one token of each of 32 sequences far into their contexts, shared key heads
        _rotate("rotate-tokens", 32, 1, 16411, 32, 8, 128, 128, "halves", True, 1, "none", False,
                "bf16", True),
        # two items' video shares, three axes (frame, row, column), a norm of each head
        _rotate("rotate-video", 2, 4388, 0, 30, 30, 64, 64, "pairs", True, 3, "none", False,
                "bf16"),
        # chunks of prompts, half of each head turned, contexts four times as long as trained; the
        # tables are made in the same pass
        _rotate("rotate-prompts", 3, 1537, 5003, 32, 8, 128, 64, "halves", False, 1, "parts", True,
                "f16", True),
        # a step of 64 sequences: 32 others are dropped and become copies of 8 running ones, all
        # get room for a token
        _step("pages-tokens", 64, 32, 2000, 1, 8, 128, 64),
        # chunks of prompts behind long contexts
        _step("pages-chunks", 8, 8, 16411, 1537, 8, 128, 64),
        # a pool with two of five pages free, packed
        _pack("pages-pack", 32, 4096, 2460, 8, 128, 64),
        # single tokens of 32 requests with adapters of their own, query, key and value at once
        _adapt("adapters-tokens", 32, 1, 1024, 3, 1024, 16, 8, "bf16"),
        # two items' video shares, query, key and value of 30 heads of 64
        _adapt("adapters-video", 2, 4388, 1920, 3, 1920, 32, 2, "bf16"),
        # ragged prompts, some without an adapter, high rank
        _adapt("adapters-prompts", 7, 2311, 4096, 1, 4096, 64, 5, "f16", True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(work(c)["flops"] for c in listed())
    most = max(work(c)["bytes"] for c in listed())
    while True:
        kind = rng.choice(["norm", "rotate", "step", "pack", "adapt"])
        batch, ragged = _log_int(rng, 1, 32), rng.random() < 0.5
        rows = 1 if rng.random() < 0.3 else _log_int(rng, 2, 4500)
        real = rng.choice(["bf16", "f16"])
        if kind == "norm":
            case = _norm("drawn", batch, rows, 8 * _log_int(rng, 8, 1024),
                         rng.choice([real, real, "f32"]), "same", rng.choice(["rms", "layer"]),
                         rng.choice(["none", "none", "rms", "layer"]), rng.random() < 0.5, ragged)
            case["stream"] = rng.choice([case["real"], "f32"])
        elif kind == "rotate":
            kv, dim = rng.randint(1, 16), rng.choice([64, 128])
            case = _rotate("drawn", batch, rows, _log_int(rng, 1, 32768) - 1,
                           kv * rng.choice([1, 1, 2, 4]), kv, dim,
                           rng.choice([dim, dim, dim // 2, 16 * rng.randint(1, dim // 16)]),
                           rng.choice(["pairs", "halves"]), rng.random() < 0.5,
                           rng.choice([1, 1, 3]),
                           rng.choice(["none", "linear", "base", "parts"]), rng.random() < 0.3,
                           rng.choice([real, real, "f32"]), ragged)
        elif kind == "step":
            case = _step("drawn", batch, rng.randint(1, 32), _log_int(rng, 2, 16384),
                         1 if rng.random() < 0.5 else _log_int(rng, 2, 2000), rng.randint(1, 24),
                         rng.choice([64, 128]), rng.choice([32, 64, 128]))
        elif kind == "pack":
            pages = _log_int(rng, 8, 8192)
            case = _pack("drawn", batch, pages, max(1, int(pages * rng.uniform(0.05, 0.98))),
                         rng.randint(1, 24), rng.choice([64, 128]), rng.choice([32, 64, 128]))
        else:
            case = _adapt("drawn", batch, rows, 8 * _log_int(rng, 16, 1024), rng.choice([1, 1, 2, 3]),
                          16 * _log_int(rng, 8, 256), 8 * rng.randint(1, 16), rng.randint(1, 12),
                          real, ragged)
        if kind in ("step", "pack") and _pool(case) * _page_bytes(case) > 3 << 30:
            continue
        w = work(case)
        if w["bytes"] <= most and w["flops"] <= top:
            del case["name"]
            return case


def _lengths(n, batch, ragged):
    """n, or ragged lengths from about half of n to n, the first the longest."""
    if not ragged:
        return [n] * batch
    return [max(1, n - int((i * 0.6180339887 % 1.0) * 0.55 * n)) for i in range(batch)]


def _page_bytes(case):
    h, d, p = case["heads"], case["dim"], case["page"]
    return h * (2 * d * p + 4 * d + 8)


def _step_lengths(case):
    """Tokens that the rows hold, which of them become children of which, and the new tokens."""
    b, f = case["batch"], case["forks"]
    held = _lengths(case["held"], b, True)
    parents = [(i // 4) % b for i in range(f)]
    held += [max(1, held[i % b] // 2) for i in range(f)]  # what the children's rows held before
    return held, parents, _lengths(case["new"], b + f, True)


def _pool(case):
    if case["kind"] == "pack":
        return case["pages"]
    held, parents, new = _step_lengths(case)
    p, b = case["page"], case["batch"]
    after = held[:b] + [held[i] for i in parents]
    return sum(-(-n // p) for n in held) + sum(-(-(n + m) // p) - n // p for n, m in zip(after, new))


def work(case):
    kind = case["kind"]
    if kind == "norm":
        t = sum(_lengths(case["rows"], case["batch"], case["ragged"]))
        c = case["cols"]
        mods = 3 * case["batch"] if case["modulated"] else 1 + (case["after"] != "none")
        return {"bytes": 2 * t * c * (SIZE[case["stream"]] + SIZE[case["real"]])
                + mods * c * SIZE[case["real"]], "flops": 10 * t * c}
    if kind == "rotate":
        t = sum(_lengths(case["rows"], case["batch"], case["ragged"]))
        h = case["heads"] + case["kv_heads"]
        table = 4 * case["turn"] * (_far(case) if case["fresh"] else t)
        return {"bytes": 2 * t * h * case["dim"] * SIZE[case["real"]] + table,
                "flops": t * h * (3 * case["turn"] + 4 * case["dim"] * case["normed"])}
    if kind == "step":
        held, parents, new = _step_lengths(case)
        p, b = case["page"], case["batch"]
        # copies: of a partly filled page all but one of those that go on behind it
        moves = sum(held[i] % p != 0 for i in parents)
        entries = sum(-(-n // p) for n in held) + 2 * sum(-(-held[i] // p) for i in parents)
        return {"bytes": 2 * moves * _page_bytes(case) + 4 * entries + 4 * _pool(case), "flops": 0}
    if kind == "pack":
        n, total = case["live"], case["pages"]
        moves = n * (total - n) / total  # of a random half-full pool
        return {"bytes": 2 * moves * _page_bytes(case) + 4 * (total + 2 * n), "flops": 0}
    t = sum(_lengths(case["rows"], case["batch"], case["ragged"]))
    n, s, r = case["slices"] * case["width"], SIZE[case["real"]], case["rank"]
    used = _adapter_of(case)
    with_one = sum(m for m, a in zip(_lengths(case["rows"], case["batch"], case["ragged"]), used)
                   if a >= 0)
    kinds = len({a for a in used if a >= 0})
    weights = kinds * r * (case["slices"] * case["cols"] + n)
    return {"bytes": s * (with_one * case["cols"] + 2 * t * n + weights),
            "flops": 2 * with_one * r * (case["slices"] * case["cols"] + n)}


def _adapter_of(case):
    """Which adapter each sequence has; every (count + 1)th has none."""
    return [i % (case["count"] + 1) - 1 if i else 0 for i in range(case["batch"])]


# ------------------------------------------------------------------ inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cumulative(lengths):
    return _ints(np.concatenate([[0], np.cumsum(lengths)]))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    make = {"norm": _prepare_norm, "rotate": _prepare_rotate, "step": _prepare_step,
            "pack": _prepare_pack, "adapt": _prepare_adapt}[case["kind"]]
    return make(case, gen, normal)


def _prepare_norm(case, gen, normal):
    lengths = _lengths(case["rows"], case["batch"], case["ragged"])
    t, c, real = sum(lengths), case["cols"], REAL[case["real"]]
    # channels of different sizes, a few large ones
    size = torch.exp(0.5 * normal(c))
    size[:: max(1, c // 7)] *= 10
    s = dict(case, offsets=_cumulative(lengths), lengths=lengths)
    s["x"] = (normal(t, c) * size + 0.3).to(REAL[case["stream"]])
    s["y"] = (normal(t, c) * 0.5).to(real)
    if case["modulated"]:
        # one projection of the conditioning gives shift, scale and gate of each item
        s["shift"], s["scale"], s["gate"] = (0.3 * normal(case["batch"], 3 * c)).to(real).chunk(3, 1)
    else:
        s["before_w"] = (1 + 0.1 * normal(c)).to(real)
        s["after_w"] = (1 + 0.1 * normal(c)).to(real)
        s["alpha"] = 0.7
    if own:
        from diffusion_activation_residual_amd import block
        weight, other = s.get("before_w"), s.get("after_w")
        s["before_n"] = block.Norm(case["before"], EPS, weight)
        s["after_n"] = None if case["after"] == "none" else block.Norm(case["after"], EPS, other)
    return s


def _far(case):
    return case["start"] + case["rows"]


def _axis_dims(case):
    if case["axes"] == 1:
        return [case["turn"]]
    first = case["turn"] // 4
    return [first, (case["turn"] - first) // 2, (case["turn"] - first) // 2]


FACTOR, TRAINED, SLOW, FAST, AMPLITUDE = 4.0, 4096, 1.0, 32.0, 1.1386


def _prepare_rotate(case, gen, normal):
    lengths = _lengths(case["rows"], case["batch"], case["ragged"])
    starts = [max(0, n - 1) for n in _lengths(case["start"] + 1, case["batch"], case["ragged"])]
    t, d, real = sum(lengths), case["dim"], REAL[case["real"]]
    h, kv = case["heads"], case["kv_heads"]
    # the rows of one projection: queries, keys, values
    qkv = normal(t, h + 2 * kv, d).to(real)
    s = dict(case, offsets=_cumulative(lengths), starts=_ints(starts), lengths=lengths,
             host_starts=starts, q=qkv[:, :h], k=qkv[:, h:h + kv])
    s["q_w"], s["k_w"] = ((1 + 0.2 * normal(d)).to(real) for _ in "qk")
    far = _far(case)
    s["places"] = None
    if case["axes"] == 3:
        # frames of rows of columns
        i = torch.arange(far, device=DEV)
        side = max(1, int(far ** 0.5 / 2))
        s["places"] = torch.stack([i // (side * side), i // side % side, i % side], 1).int()
    if not case["fresh"]:
        s["cos"], s["sin"] = _plain_table(s)
    if own and not case["fresh"]:
        from diffusion_activation_residual_amd import kv8
        s["turned"] = kv8.Rotation(s["cos"], s["sin"], interleaved=case["layout"] == "pairs")
    return s


def _prepare_pool(case, gen):
    pool, h, d, p = _pool(case), case["heads"], case["dim"], case["page"]

    def codes(*shape):
        return torch.randint(-127, 128, shape, generator=gen, device=DEV, dtype=torch.int8)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    s = dict(case, pool=pool, k=codes(pool, h, p, d), v=codes(pool, h, d, p),
             k_scale=0.02 + 0.02 * rand(pool, h), v_scale=0.02 + 0.02 * rand(pool, h),
             k_mean=rand(pool, h, d) - 0.5)
    if own:
        from diffusion_activation_residual_amd import kv8
        s["cache"] = kv8.Cache.over(s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_mean"])
    return s


def _prepare_step(case, gen, normal):
    s = _prepare_pool(case, gen)
    held, parents, new = _step_lengths(case)
    b, f, p = case["batch"], case["forks"], case["page"]
    per = [-(-n // p) for n in held]
    width = max(-(-(n + max(new)) // p) for n in held) + 1
    order = torch.randperm(s["pool"], generator=gen, device=DEV).cpu().numpy()
    table = np.full((b + f, width), -1, np.int64)
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    refs = np.bincount(table[table >= 0], minlength=s["pool"])
    # table, lengths and reference counts in one piece: a pass starts from a copy of it
    s["meta"] = _ints(np.concatenate([table.reshape(-1), held, refs]))
    s.update(width=width, rows=b + f, parents=_ints(parents), children=_ints(range(b, b + f)),
             new=_ints(new), most=max(new))
    return s


def _prepare_pack(case, gen, normal):
    s = _prepare_pool(case, gen)
    b, n = case["batch"], case["live"]
    order = torch.randperm(s["pool"], generator=gen, device=DEV).cpu().numpy()[:n]
    width = -(-n // b) + 2
    table = np.full((b, width), -1, np.int64)
    for i, part in enumerate(np.array_split(order, b)):
        table[i, :len(part)] = part
    # the second half of the sequences shares its first page with the first half
    for i in range(b // 2, b):
        if i > 0 and table[i, 0] >= 0 and table[i - b // 2, 0] >= 0:
            table[i, width - 1] = table[i - b // 2, 0]
    refs = np.bincount(table[table >= 0], minlength=s["pool"])
    lengths = (table >= 0).sum(1) * case["page"]
    s["meta"] = _ints(np.concatenate([table.reshape(-1), lengths, refs]))
    s.update(width=width, rows=b)
    return s


def _prepare_adapt(case, gen, normal):
    lengths = _lengths(case["rows"], case["batch"], case["ragged"])
    t, k, n, r = sum(lengths), case["cols"], case["slices"] * case["width"], case["rank"]
    real = REAL[case["real"]]
    s = dict(case, lengths=lengths, offsets=_cumulative(lengths), most=max(lengths),
             host_ids=_adapter_of(case), ids=_ints(_adapter_of(case)))
    s["x"] = normal(t, k).to(real)
    s["y"] = normal(t, n).to(real)
    s["a"] = (normal(case["count"], case["slices"] * r, k) * k ** -0.5).to(real)
    s["b"] = (normal(case["count"], n, r) * r ** -0.5).to(real)
    s["scales"] = 0.5 + torch.rand(case["count"], generator=gen, device=DEV)
    if own:
        from diffusion_activation_residual_amd import block
        s["adapters"] = block.Adapters(s["a"], s["b"], s["scales"], slices=case["slices"])
    return s


# ------------------------------------------------------------------ the operators

def run(state):
    if own:
        return _OWN[state["kind"]](state)
    return _PLAIN[state["kind"]](state)


def _own_norm(s):
    from diffusion_activation_residual_amd import block
    if s["modulated"]:
        return block.residual_norm(s["x"], s["y"], before=s["before_n"], after=s["after_n"],
                                   gate=s["gate"], scale=s["scale"], shift=s["shift"],
                                   offsets=s["offsets"])
    return block.residual_norm(s["x"], s["y"], before=s["before_n"], after=s["after_n"],
                               gate_scale=s["alpha"])


def _own_rotate(s):
    from diffusion_activation_residual_amd import block
    if s["fresh"]:
        turned = block.rotation_table(
            s["turn"], rows=None if s["axes"] > 1 else _far(s), positions=s["places"],
            axis_dims=_axis_dims(s), scaling=s["scaling"], factor=FACTOR, trained=TRAINED,
            slow=SLOW, fast=FAST, amplitude=AMPLITUDE, interleaved=s["layout"] == "pairs",
            device=s["q"].device)
    else:
        turned = s["turned"]
    out = block.rotate([s["q"], s["k"]], turned, s["offsets"], s["starts"],
                       weights=[s["q_w"], s["k_w"]] if s["normed"] else None, eps=EPS)
    return (turned.cos, turned.sin, *out) if s["fresh"] else tuple(out)


def _parts(s):
    """A copy of table, lengths and reference counts."""
    meta = s["meta"].clone()
    n = s["rows"] * s["width"]
    return meta[:n].view(s["rows"], s["width"]), meta[n:n + s["rows"]], meta[n + s["rows"]:]


def _own_step(s):
    from diffusion_activation_residual_amd import kv8
    pages = kv8.Pages(*_parts(s), page_tokens=s["page"])
    pages.free(s["children"])
    pages.fork(s["parents"], s["children"])
    moves, missing = pages.reserve(s["new"], s["most"])
    s["cache"].copy(moves)
    return (pages.table, pages.lengths, pages.refs, moves.source, moves.target, missing, s["k"],
            s["v"], s["k_scale"], s["v_scale"], s["k_mean"])


def _own_pack(s):
    from diffusion_activation_residual_amd import kv8
    pages = kv8.Pages(*_parts(s), page_tokens=s["page"])
    moves, live = pages.compact()
    s["cache"].copy(moves)
    return (pages.table, pages.refs, live, s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_mean"])


def _own_adapt(s):
    return s["adapters"].add(s["x"], s["y"], s["ids"], s["offsets"], s["most"])


_OWN = {"norm": _own_norm, "rotate": _own_rotate, "step": _own_step, "pack": _own_pack,
        "adapt": _own_adapt}


def _normalise(v, kind, weight):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v if weight is None else v * weight.float()


def _plain_norm(s):
    x, b = s["x"].float(), s["y"].float()
    if s["after"] != "none":
        b = _normalise(b, s["after"], s.get("after_w"))
    if s["modulated"]:
        counts = torch.tensor(s["lengths"], device=DEV)
        shift, scale, gate = (torch.repeat_interleave(s[w].float(), counts, 0)
                              for w in ("shift", "scale", "gate"))
        r = x + gate * b
        h = _normalise(r, s["before"], None) * (1 + scale) + shift
    else:
        r = x + s["alpha"] * b
        h = _normalise(r, s["before"], s["before_w"])
    return r.to(s["x"].dtype), h.to(s["y"].dtype)


def _plain_table(s):
    """Cosines and sines of the angles, in 64 bits: far positions turn many times."""
    columns = []
    for axis, dim in enumerate(_axis_dims(s)):
        base = 10000.0
        if s["scaling"] == "base":
            base *= FACTOR ** (dim / (dim - 2))
        speed = base ** (-torch.arange(0, dim, 2, device=DEV, dtype=torch.float64) / dim)
        if s["scaling"] == "linear":
            speed = speed / FACTOR
        elif s["scaling"] == "parts":
            turns = TRAINED * speed / (2 * math.pi)
            keep = ((turns - SLOW) / (FAST - SLOW)).clamp(0, 1)
            speed = speed * (keep + (1 - keep) / FACTOR)
        place = torch.arange(_far(s), device=DEV) if s["places"] is None else s["places"][:, axis]
        columns.append(place.double()[:, None] * speed)
    angle = torch.cat(columns, 1)
    return (AMPLITUDE * angle.cos()).float(), (AMPLITUDE * angle.sin()).float()


def _plain_rotate(s):
    cos, sin = _plain_table(s) if s["fresh"] else (s["cos"], s["sin"])
    place = torch.cat([torch.arange(a, a + n, device=DEV)
                       for a, n in zip(s["host_starts"], s["lengths"])])
    c, w, half = cos[place][:, None], sin[place][:, None], s["turn"] // 2
    out = []
    for x, weight in ((s["q"], s["q_w"]), (s["k"], s["k_w"])):
        y = x.float()
        y = _normalise(y, "rms", weight) if s["normed"] else y.clone()
        one = slice(0, 2 * half, 2) if s["layout"] == "pairs" else slice(0, half)
        two = slice(1, 2 * half, 2) if s["layout"] == "pairs" else slice(half, 2 * half)
        a, b = y[..., one], y[..., two]
        y[..., one], y[..., two] = a * c - b * w, a * w + b * c
        out.append(y.to(x.dtype))
    return (cos, sin, *out) if s["fresh"] else tuple(out)


def _named(refs, names):
    """How often each page is named."""
    return torch.bincount(names.long(), minlength=refs.numel()).to(torch.int32)


def _plain_step(s):
    table, lengths, refs = _parts(s)
    p, width = s["page"], s["width"]
    children, parents = s["children"].long(), s["parents"].long()
    # dropped
    names = table[children]
    refs -= _named(refs, names[names >= 0])
    table[children] = -1
    # forked
    entry = torch.arange(width, device=DEV)
    own_pages = (lengths[parents] + p - 1).div(p, rounding_mode="floor")
    names = torch.where(entry < own_pages[:, None], table[parents], -1)
    table[children] = names
    lengths[children] = lengths[parents]
    refs += _named(refs, names[names >= 0])
    # room for the new tokens
    new = s["new"]
    first = lengths.div(p, rounding_mode="floor")
    last = (lengths + new + p - 1).div(p, rounding_mode="floor").clamp(max=width)
    written = (entry >= first[:, None]) & (entry < last[:, None]) & (new > 0)[:, None]
    place = torch.arange(table.numel(), device=DEV).view_as(table)
    held = written & (table >= 0)
    writers = _named(refs, table[held])
    keeper = torch.full((s["pool"],), table.numel(), device=DEV)
    keeper.scatter_reduce_(0, table[held].long(), place[held], "amin")
    at = table.clamp(min=0).long()
    shared = held & (refs[at] > 1)
    kept = shared & (refs[at] <= writers[at]) & (keeper[at] == place)
    need = written & ((table < 0) | (shared & ~kept))
    spare = torch.nonzero(refs == 0)[:, 0]
    wanted = int(need.sum())
    missing = max(0, wanted - spare.numel())
    source, target = (torch.full_like(lengths, -1) for _ in range(2))
    if not missing:
        fresh = spare[:wanted].to(torch.int32)
        old = table[need]
        table[need] = fresh
        refs -= _named(refs, old[old >= 0])
        refs[fresh.long()] = 1
        moved = torch.nonzero(need)
        begun = (old >= 0) & (moved[:, 1] == first[moved[:, 0]]) & (lengths[moved[:, 0]] % p != 0)
        source[moved[begun, 0]], target[moved[begun, 0]] = old[begun], fresh[begun]
        for t in ("k", "v", "k_scale", "v_scale", "k_mean"):
            s[t][fresh[begun].long()] = s[t][old[begun].long()]
    return (table, lengths, refs, source, target,
            torch.tensor([missing], dtype=torch.int32, device=DEV), s["k"], s["v"], s["k_scale"],
            s["v_scale"], s["k_mean"])


def _plain_pack(s):
    table, _, refs = _parts(s)
    used = refs > 0
    live = int(used.sum())
    target = torch.nonzero(~used[:live])[:, 0]
    # the highest page goes to the lowest free one
    source = torch.nonzero(used)[:, 0].flip(0)[:target.numel()]
    where = torch.arange(s["pool"], device=DEV, dtype=torch.int32)
    where[source] = target.to(torch.int32)
    table = torch.where(table >= 0, where[table.clamp(min=0).long()], table)
    refs[target], refs[source] = refs[source], 0
    for t in ("k", "v", "k_scale", "v_scale", "k_mean"):
        s[t][target] = s[t][source]
    return (table, refs, torch.tensor([live], dtype=torch.int32, device=DEV), s["k"], s["v"],
            s["k_scale"], s["v_scale"], s["k_mean"])


def _plain_adapt(s):
    out, r, at = s["y"].float(), s["rank"], 0
    for i, n in enumerate(s["lengths"]):
        a = s["host_ids"][i]
        if a >= 0:
            low = s["x"][at:at + n].float() @ s["a"][a].float().t()
            for j in range(s["slices"]):
                cols = slice(j * s["width"], (j + 1) * s["width"])
                up = low[:, j * r:(j + 1) * r] @ s["b"][a, cols].float().t()
                out[at:at + n, cols] += s["scales"][a] * up
        at += n
    return out.to(s["y"].dtype)


_PLAIN = {"norm": _plain_norm, "rotate": _plain_rotate, "step": _plain_step, "pack": _plain_pack,
          "adapt": _plain_adapt}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotate": _exact_rotate, "step": _exact_step,
            "pack": _exact_pack, "adapt": _exact_adapt}[case["kind"]](s)


def _exact_norm(s):
    def norm(v, kind, weight):
        n = v.shape[1]
        mean = v.sum(1) / n if kind == "layer" else torch.zeros_like(v[:, 0])
        var = ((v - mean[:, None]) ** 2).sum(1) / n
        v = (v - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
        return v if weight is None else v * weight.double()

    first, second, at = [], [], 0
    for i, n in enumerate(s["lengths"]):
        x, y = s["x"][at:at + n].double(), s["y"][at:at + n].double()
        at += n
        if s["after"] != "none":
            y = norm(y, s["after"], s.get("after_w"))
        r = x + y * (s["gate"][i].double() if s["modulated"] else s["alpha"])
        h = norm(r, s["before"], s.get("before_w"))
        if s["modulated"]:
            h = h + h * s["scale"][i].double() + s["shift"][i].double()
        first.append(r)
        second.append(h)
    return torch.cat(first), torch.cat(second)


def _exact_rotate(s):
    outputs = []
    if s["fresh"]:
        columns = []
        for axis, dim in enumerate(_axis_dims(s)):
            for pair in range(dim // 2):
                speed = math.exp(-2 * pair / dim * math.log(
                    1e4 * (FACTOR ** (dim / (dim - 2)) if s["scaling"] == "base" else 1)))
                if s["scaling"] == "linear":
                    speed /= FACTOR
                if s["scaling"] == "parts":
                    turns = TRAINED / (2 * math.pi / speed)
                    keep = min(1.0, max(0.0, (turns - SLOW) / (FAST - SLOW)))
                    speed = keep * speed + (1 - keep) * speed / FACTOR
                if s["places"] is None:
                    place = torch.arange(_far(s), device=DEV, dtype=torch.float64)
                else:
                    place = s["places"][:, axis].double()
                columns.append(place * speed)
        angle = torch.stack(columns, 1)
        cos, sin = AMPLITUDE * torch.cos(angle), AMPLITUDE * torch.sin(angle)
        outputs = [cos, sin]
        # the rotation's definition takes the tables as they are held
        cos, sin = cos.float().double(), sin.float().double()
    else:
        cos, sin = s["cos"].double(), s["sin"].double()
    for x, weight in ((s["q"], s["q_w"]), (s["k"], s["k_w"])):
        rows, at = [], 0
        for start, n in zip(s["host_starts"], s["lengths"]):
            y = x[at:at + n].double()
            at += n
            if s["normed"]:
                y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / s["dim"] + EPS) * weight.double()
            # as a product with complex numbers
            turn = torch.complex(cos[start:start + n], sin[start:start + n])[:, None]
            m = turn.shape[-1]
            z = y[..., :2 * m]
            z = z.unflatten(-1, (m, 2)) if s["layout"] == "pairs" else \
                z.unflatten(-1, (2, m)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z if s["layout"] == "pairs" else z.transpose(-1, -2)
            rows.append(torch.cat([z.flatten(-2), y[..., 2 * m:]], -1))
        outputs.append(torch.cat(rows))
    return tuple(outputs)


def _moved(s, pairs):
    """The cache's buffers after copying pages, one pair after another."""
    out = []
    for t in ("k", "v", "k_scale", "v_scale", "k_mean"):
        buffer = s[t].clone() if s[t].dtype == torch.int8 else s[t].double()
        for a, b in pairs:
            buffer[b] = buffer[a]
        out.append(buffer)
    return out


def _lists(s):
    meta = s["meta"].tolist()
    n, w = s["rows"] * s["width"], s["width"]
    table = [meta[i * w:(i + 1) * w] for i in range(s["rows"])]
    return table, meta[n:n + s["rows"]], meta[n + s["rows"]:]


def _exact_step(s):
    table, lengths, refs = _lists(s)
    p = s["page"]
    parents, children, new = s["parents"].tolist(), s["children"].tolist(), s["new"].tolist()
    for c in children:
        for page in table[c]:
            if page >= 0:
                refs[page] -= 1
        table[c] = [-1] * s["width"]
    for a, c in zip(parents, children):
        lengths[c] = lengths[a]
        for e in range(-(-lengths[a] // p)):
            table[c][e] = table[a][e]
            refs[table[a][e]] += 1
    places = [(i, e) for i, n in enumerate(lengths)
              for e in range(n // p, min(s["width"], -(-(n + new[i]) // p)))]
    writers = {}
    for i, e in places:
        writers.setdefault(table[i][e], []).append((i, e))
    need = []
    for i, e in places:
        page = table[i][e]
        if page < 0 or (refs[page] > 1 and not (refs[page] <= len(writers[page])
                                                and writers[page][0] == (i, e))):
            need.append((i, e))
    spare = [q for q, n in enumerate(refs) if n == 0]
    missing = max(0, len(need) - len(spare))
    source, target, pairs = [-1] * s["rows"], [-1] * s["rows"], []
    if not missing:
        for (i, e), q in zip(need, spare):
            page = table[i][e]
            table[i][e], refs[q] = q, 1
            if page >= 0:
                refs[page] -= 1
                if e == lengths[i] // p and lengths[i] % p:
                    source[i], target[i] = page, q
                    pairs.append((page, q))
    return (_ints(table), _ints(lengths), _ints(refs), _ints(source), _ints(target),
            _ints([missing]), *_moved(s, pairs))


def _exact_pack(s):
    table, _, refs = _lists(s)
    live = sum(n > 0 for n in refs)
    low = [q for q in range(live) if refs[q] == 0]
    high = [q for q in range(len(refs) - 1, live - 1, -1) if refs[q] > 0]
    to = dict(zip(high, low))
    for a, b in to.items():
        refs[a], refs[b] = 0, refs[a]
    table = [[to.get(q, q) for q in row] for row in table]
    return (_ints(table), _ints(refs), _ints([live]), *_moved(s, list(to.items())))


def _exact_adapt(s):
    rows, at = [], 0
    for n, a in zip(s["lengths"], s["host_ids"]):
        x, y = s["x"][at:at + n].double(), s["y"][at:at + n].double()
        at += n
        if a >= 0:
            # the adapter as the matrix that it stands for, a slice of columns at a time
            down = s["a"][a].double().view(s["slices"], s["rank"], -1)
            up = s["b"][a].double().view(s["slices"], s["width"], -1)
            whole = torch.cat([u @ d for u, d in zip(up, down)])
            y = y + s["scales"][a].double() * (x @ whole.t().contiguous())
        rows.append(y)
    return torch.cat(rows)
