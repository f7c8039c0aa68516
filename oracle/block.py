"""Plain 64-bit models (numpy, no GPU) of cfz_residual_norm, cfz_rotation_table, cfz_rotate and
cfz_adapters_add, and bounds on how far fp32 arithmetic may be from them.

Bounds count roundings, U = 2^-24 each (half a step of fp32).  A sum over a row adds at most 64 values
in a thread and then 8 levels across threads: within 72 U of the sum of magnitudes, 75 with the
division by n.  So a mean is off by at most 75 U mean|v|; a deviation d = v - mean by e = e_in +
75 U mean|v| + U |d|; the square root of the mean square by the root mean square of e plus 40 U of
itself (half of the sum's 75 and the additions); the quotient's rounding and the product with it add 3 U."""
import numpy as np

U = 2.0 ** -24


def normalise(v, kind, eps, weight=None, bias=None, e_in=0.0):
    """(norm of the rows of v, bound of its error for inputs off by e_in)."""
    v = np.asarray(v, np.float64)
    e = np.broadcast_to(np.asarray(e_in, np.float64), v.shape)
    if kind == "none":
        return v, e
    mean = v.mean(-1, keepdims=True) if kind == "layer" else np.zeros_like(v[..., :1])
    d = v - mean
    if kind == "layer":
        e = e + e.mean(-1, keepdims=True) + 75 * U * np.abs(v).mean(-1, keepdims=True)
    e = e + U * np.abs(d)
    root = np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    e_root = np.sqrt((e * e).mean(-1, keepdims=True)) + 42 * U * root
    with np.errstate(divide="ignore", invalid="ignore"):
        out = d / root
        off = (e + np.abs(out) * e_root) / root + 3 * U * np.abs(out)
    if weight is not None:
        out, off = out * weight, (off + U * np.abs(out)) * np.abs(weight)
    if bias is not None:
        out = out + bias
        off = off + U * np.abs(out)
    return out, off


def residual_norm(x, y=None, gate=None, gate_scale=1.0, after=None, before=None, scale=None,
                  shift=None):
    """Rows of one item: (r, h, bound of r, bound of h), before the rounding of the results."""
    x = np.asarray(x, np.float64)
    r, e = x, np.zeros_like(x)
    if y is not None:
        b, e = normalise(y, **(after or {"kind": "none", "eps": 0.0}))
        g = gate_scale * (1.0 if gate is None else np.asarray(gate, np.float64))
        r = x + g * b
        e = np.abs(g) * (e + U * np.abs(b)) + U * np.abs(r) + U * np.abs(g * b)
    h, off = normalise(r, **(before or {"kind": "none", "eps": 0.0}), e_in=e)
    if scale is not None:
        s = 1.0 + np.asarray(scale, np.float64)
        off = np.abs(s) * off + 2 * U * np.abs(h * s)
        h = h * s
    if shift is not None:
        h = h + np.asarray(shift, np.float64)
        off = off + U * np.abs(h)
    return r, h, e, off


def rotation_table(axis_dims, positions, base=10000.0, scaling="none", factor=1.0, trained=0,
                   slow=1.0, fast=32.0, amplitude=1.0):
    """(cos, sin, angle) [rows, pairs]; positions [rows, axes]."""
    speeds, axis = [], []
    for j, d in enumerate(axis_dims):
        b = base * factor ** (d / (d - 2)) if scaling == "base" else base
        for i in range(d // 2):
            s = b ** (-2 * i / d)
            if scaling == "linear":
                s /= factor
            if scaling == "parts":
                n = trained * s / (2 * np.pi)
                k = min(1.0, max(0.0, (n - slow) / (fast - slow)))
                s = s * k + s * (1 - k) / factor
            speeds.append(s)
            axis.append(j)
    angle = np.asarray(positions, np.float64)[:, axis] * np.array(speeds)
    return amplitude * np.cos(angle), amplitude * np.sin(angle), angle


def rotate(x, cos, sin, interleaved, normed=False, eps=0.0, weight=None):
    """x [tokens, heads, dim]; cos, sin [tokens, rot / 2] of the tokens' positions, or None:
    (result, bound of its error)."""
    x = np.asarray(x, np.float64)
    off = np.zeros_like(x)
    if normed:
        x, off = normalise(x, "rms", eps, weight)
        off = off + 2 * U * np.abs(x)
    if cos is None:
        return x, off
    half = cos.shape[-1]
    i = np.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos[:, None, :].astype(np.float64), sin[:, None, :].astype(np.float64)
    y, e = x.copy(), off.copy()
    with np.errstate(invalid="ignore"):
        a, b, ea, eb = x[..., one], x[..., two], off[..., one], off[..., two]
        y[..., one], y[..., two] = a * c - b * s, a * s + b * c
        e[..., one] = np.abs(c) * ea + np.abs(s) * eb + 2 * U * (np.abs(a * c) + np.abs(b * s))
        e[..., two] = np.abs(s) * ea + np.abs(c) * eb + 2 * U * (np.abs(a * s) + np.abs(b * c))
    return y, e


def adapters_add(x, y, a, b, scale, slices, half):
    """Rows of one sequence with adapter a [slices * rank, cols_in], b [cols_out, rank] in 16 bits:
    (y + scale (x a^T) b^T, bound of its error before the rounding of the result).

    The products of 16-bit numbers are exact in fp32, so that a sum of n of them in any order is within 2 n U
    of the sum of magnitudes (two roundings a term); h = scale x a^T takes three more roundings
    and is then split: `half` ("bf16": 2^-16 of itself, "f16": 2^-21 of its row's largest)."""
    x, y, a, b = (np.asarray(t, np.float64) for t in (x, y, a, b))
    rank = b.shape[1]
    h = scale * (x @ a.T)
    e = abs(scale) * 2 * (x.shape[1] + 16) * U * (np.abs(x) @ np.abs(a).T) + 3 * U * np.abs(h)
    out, off, at = y.copy(), np.zeros_like(y), 0
    for i, n in enumerate(slices):
        r, c = slice(i * rank, (i + 1) * rank), slice(at, at + n)
        at += n
        top = np.abs(h[:, r]) if half == "bf16" else np.abs(h[:, r]).max(-1, keepdims=True)
        eh = e[:, r] + (2.0 ** -16 if half == "bf16" else 2.0 ** -21) * (top + e[:, r])
        w = np.abs(b[c]).T
        out[:, c] += h[:, r] @ b[c].T
        off[:, c] = eh @ w + 4 * (rank + 8) * U * ((np.abs(h[:, r]) + eh) @ w) + \
            U * np.abs(out[:, c])
    return out, off
