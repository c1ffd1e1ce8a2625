"""8-bit matrices with a power-of-two scale per group of 128 and what is computed with them, float64
(oracle).

    value = q 2^(s - 127),  s the least byte for which the group's largest finite magnitude is within
    the type's range, q rounded to nearest even; infinities and NaN become NaN
Groups: "row" (128 of a row), "col" (128 of a column), "tile" (128 x 128).
"""

from __future__ import annotations

import numpy as np

GROUP = 128
# type: (explicit significand bits, least normal exponent, largest value)
TYPES = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}


def f64(a):
    return np.asarray(a, dtype=np.float64)


def scale_shape(rows, cols, groups):
    up = lambda n: -(-n // GROUP)  # noqa: E731
    return (rows if groups == "row" else up(rows), cols if groups == "col" else up(cols))


def spread(s, rows, cols, groups):
    """One entry per element from one per group."""
    i, j = np.arange(rows), np.arange(cols)
    return np.asarray(s)[np.ix_(i if groups == "row" else i // GROUP,
                                j if groups == "col" else j // GROUP)]


def round_to(u, kind):
    """Nearest value of the type (ties to the even significand); the caller stays in range."""
    bits, least, _ = TYPES[kind]
    u = f64(u)
    _, e = np.frexp(np.abs(u))
    step = np.exp2(np.maximum(e - 1, least).astype(np.float64) - bits)
    return np.rint(u / step) * step


def quantize(x, groups, kind):
    """(q, s): the 8-bit values before scaling, and the scales' bytes."""
    x = f64(x)
    rows, cols = x.shape
    x = np.where(np.isfinite(x), x, np.nan)
    a = np.nan_to_num(np.abs(x))
    gr, gc = scale_shape(rows, cols, groups)
    pad = np.zeros((gr * GROUP if groups != "row" else rows,
                    gc * GROUP if groups != "col" else cols))
    pad[:rows, :cols] = a
    top = pad.reshape(gr, pad.shape[0] // max(gr, 1), gc, -1).max(axis=(1, 3))
    big = TYPES[kind][2]
    s = np.zeros(top.shape, dtype=np.int64)
    for _ in range(255):                       # the least byte that is large enough
        s += top > big * np.exp2(s - 127.0)
    return round_to(x / np.exp2(spread(s, rows, cols, groups) - 127.0), kind), s


def values(q, s, groups):
    q = f64(q)
    v = np.where(np.asarray(s) == 255, np.nan, np.exp2(f64(s) - 127.0))
    return q * spread(v, *q.shape, groups)


def _gelu(gate):
    """((1 + tanh u) / 2, du/dgate), u = sqrt(2 / pi) (gate + 0.044715 gate^3); the first as
    1 / (1 + exp(-2 u)), which has no cancellation where it is small."""
    c = np.sqrt(2 / np.pi)
    with np.errstate(over="ignore"):
        p = 1 / (1 + np.exp(-2 * c * (gate + 0.044715 * gate ** 3)))
    return p, c * (1 + 3 * 0.044715 * gate ** 2)


def activation(kind, gate, up):
    """SwiGLU gate sigmoid(gate) up, or GELU (tanh form) of gate."""
    gate = f64(gate)
    if kind == "swiglu":
        return gate / (1 + np.exp(-gate)) * f64(up)
    return gate * _gelu(gate)[0]


def activation_grads(kind, dy, gate, up):
    """(dgate, dup)."""
    dy, gate = f64(dy), f64(gate)
    if kind == "swiglu":
        p = 1 / (1 + np.exp(-gate))
        return dy * f64(up) * p * (1 + gate * (1 - p)), dy * gate * p
    p, slope = _gelu(gate)
    return dy * (p + gate * 2 * p * (1 - p) * slope), None
