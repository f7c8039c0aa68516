"""Plain 64-bit model of the 8-bit paged K/V cache (numpy, no GPU): what cfz_kv8_append, _gather,
_attend and _select compute, written token by token from their definitions."""
import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0}


def e4m3_values():
    """The value of each of the 128 non-negative bytes (the last is NaN)."""
    out = np.empty(128)
    for byte in range(128):
        exp, man = byte >> 3, byte & 7
        out[byte] = man * 2.0 ** -9 if exp == 0 else (8 + man) * 2.0 ** (exp - 10)
    out[127] = np.nan
    return out


_GRID = e4m3_values()[:127]


def nearest(y, fmt):
    """The code value nearest to y (ties to the even code), saturating; NaN gives 0."""
    y = np.nan_to_num(np.asarray(y, np.float64), nan=0.0, posinf=1e30, neginf=-1e30)
    y = np.clip(y, -QMAX[fmt], QMAX[fmt])
    if fmt == "int8":
        return np.rint(y) + 0.0
    mid = (_GRID[1:] + _GRID[:-1]) / 2
    a = np.abs(y)
    i = np.searchsorted(mid, a)  # the first border >= a
    tie = (i < len(mid)) & (a == mid[np.minimum(i, len(mid) - 1)])
    i = i + (tie & (i % 2 == 1))
    return np.copysign(_GRID[i], y)  # e4m3 keeps the sign of a zero


def code_bytes(values, fmt):
    """The bytes that hold code values."""
    v = np.asarray(values, np.float64)
    if fmt == "int8":
        return v.astype(np.int8).view(np.uint8)
    i = np.searchsorted(_GRID, np.abs(v))
    return (i + 128 * np.signbit(v)).astype(np.uint8)


def rotate(x, cos, sin, interleaved):
    """x [heads, dim]; cos, sin [rot / 2]."""
    y = np.array(x, np.float64)
    h = len(cos)
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        c, s = float(cos[i]), float(sin[i])
        with np.errstate(invalid="ignore"):
            y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, a] * s + x[:, b] * c
    return y


class Pool:
    """Code values (token-major) and fp32 scales of a pool of pages."""

    def __init__(self, pages, heads, dim, page, fmt):
        self.pages, self.heads, self.dim, self.page, self.fmt = pages, heads, dim, page, fmt
        self.k = np.zeros((pages, heads, page, dim))
        self.v = np.zeros((pages, heads, page, dim))
        self.ks = np.zeros((pages, heads), np.float32)
        self.vs = np.zeros((pages, heads), np.float32)
        self.km = np.zeros((pages, heads, dim), np.float32)

    def page_of(self, table, i):
        """The pool page of logical page i, or None."""
        if not 0 <= i < len(table):
            return None
        p = int(table[i])
        return p if 0 <= p < self.pages else None

    def append(self, k, v, table, old, rotation=None, positions=None):
        """Token rows k, v [n, heads, dim] (float64) behind `old` tokens of one sequence."""
        room = len(table) * self.page
        old = min(max(old, 0), room)
        n = min(len(k), room - old)
        k, v = np.array(k[:n], np.float64), np.array(v[:n], np.float64)
        if rotation is not None:
            cos, sin, inter = rotation
            for t in range(n):
                pos = old + t if positions is None else int(positions[t])
                pos = min(max(pos, 0), len(cos) - 1)
                k[t] = rotate(k[t], cos[pos], sin[pos], inter)
        for j in range(old // self.page, -(-(old + n) // self.page)):
            lo, hi = max(old, j * self.page), min(old + n, (j + 1) * self.page)
            if hi <= lo:
                continue
            page = self.page_of(table, j)
            if page is None:
                continue
            keep = lo - j * self.page
            for h in range(self.heads):
                for new, codes, scales in ((k, self.k, self.ks), (v, self.v, self.vs)):
                    x = new[lo - old:hi - old, h]
                    size = np.abs(np.where(np.isfinite(x), x, 0.0)).max()
                    prior = scales[page, h] if keep else np.float32(0)
                    s = max(prior, np.float32(size / QMAX[self.fmt]))
                    held = codes[page, h]
                    with np.errstate(divide="ignore", invalid="ignore"):
                        if keep and s > prior:
                            held[:keep] = nearest(held[:keep] * np.float64(prior) / np.float64(s),
                                                  self.fmt)
                        fresh = nearest(x / np.float64(s), self.fmt) if s > 0 else np.zeros_like(x)
                    held[keep:keep + hi - lo] = fresh
                    scales[page, h] = s
                live = self.k[page, h, :keep + hi - lo]
                self.km[page, h] = live.mean(0) * np.float64(self.ks[page, h])

    def dense(self, table, head, lo, hi):
        """Keys and values [hi - lo, dim] of tokens lo .. hi, and which of them exist."""
        k, v = np.zeros((hi - lo, self.dim)), np.zeros((hi - lo, self.dim))
        live = np.zeros(hi - lo, bool)
        for t in range(lo, hi):
            page = self.page_of(table, t // self.page)
            if page is not None:
                k[t - lo] = self.k[page, head, t % self.page] * np.float64(self.ks[page, head])
                v[t - lo] = self.v[page, head, t % self.page] * np.float64(self.vs[page, head])
                live[t - lo] = True
        return k, v, live

    def attend(self, q, table, length, causal, scale, lists=None, q_block=1):
        """One sequence: q [n, q_heads, dim] -> out, lse, and for error bounds sum w |v| and the
        largest sum |q k| of each row."""
        n, q_heads, _ = q.shape
        length = min(max(length, 0), len(table) * self.page)
        group = q_heads // self.heads
        out, size = np.zeros(q.shape), np.zeros(q.shape)
        lse, reach = np.full((n, q_heads), -np.inf), np.zeros((n, q_heads))
        for head in range(self.heads):
            k, v, live = self.dense(table, head, 0, length)
            at = np.arange(length)
            for i in range(n):
                see = live & (at <= length - n + i) if causal else live.copy()
                if lists is not None:
                    see &= np.isin(at // self.page, lists[i // q_block, head])
                if not see.any():
                    continue
                for h in range(head * group, (head + 1) * group):
                    s = scale * (k[see] @ q[i, h])
                    top = s.max()
                    w = np.exp(s - top)
                    out[i, h] = w @ v[see] / w.sum()
                    size[i, h] = w @ np.abs(v[see]) / w.sum()
                    lse[i, h] = top + np.log(w.sum())
                    reach[i, h] = scale * (np.abs(k[see]) @ np.abs(q[i, h])).max()
        return out, lse, size, reach

    def select(self, q, table, length, causal, q_block, count, first, last):
        """One sequence: lists [ceil(n / q_block), heads, count]."""
        n, q_heads, _ = q.shape
        length = min(max(length, 0), len(table) * self.page)
        group = q_heads // self.heads
        units = -(-n // q_block)
        lists = np.full((units, self.heads, count), -1, np.int32)
        for u in range(units):
            stop = min(n, (u + 1) * q_block)
            end = length - n + stop if causal else length
            seen = max(0, -(-end // self.page))
            for h in range(self.heads):
                x = q[u * q_block:stop, h * group:(h + 1) * group].sum((0, 1))
                ranked = []
                for p in range(seen):
                    page = self.page_of(table, p)
                    if page is None:
                        continue
                    s = float(self.km[page, h].astype(np.float64) @ x)
                    kept = p < first or p >= seen - last
                    low = np.isnan(s)
                    ranked.append((not kept, low, 0.0 if low else -s, p))
                picked = sorted(p for *_, p in sorted(ranked)[:count])
                lists[u, h, :len(picked)] = picked
        return lists
