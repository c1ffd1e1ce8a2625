"""Norms with a residual and activations with 8-bit results and checkpoints, against the float64 oracle.

Elementwise, u = 2^-24.  Norms as in the plain norm's tests: a row's sums are within 64 u of their sums of
absolute values, and h = x + r is rounded once, so with A = (|h| + mean|h|) rstd
    |dy|  <= 66 u (A |w| + |b|),
    |ddx| <= 66 u rstd (|g| + mean|g| + A mean(|g| A)) + 2 u |dres|,
    |ddw| <= (66 + rows) u sum |dy| A,  |ddb| <= (66 + rows) u sum |dy|.
Activations: exp and the division are the special-function unit's, (2 + 1.2 |a|) 2^-23 and 2^-22 relative,
with an argument a that has four roundings in GELU, so p = 1 / (1 + exp(-a)) is within
T = ((4 + 4 |a|) (1 - p) + 6) 2^-23 of itself, and what is made of it within T and some u per operation.

A stored result is rounded once: bf16 2^-8 of it; in 8 bits half a step of the stored value, 2^-4 (e4m3) or
2^-3 (e5m2) of it or half of the least step, and the scale is that of a largest value within the error.
"""

import numpy as np
import pytest
import torch

from oracle import fp8 as o8
from oracle import norm as onorm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _empty8(rows, cols, kind="e4m3", groups=0, extra=0):
    from matrix_optimizer_owner_gb300 import mfsdp
    pitch = -(-cols // 16) * 16 + 16 * extra
    data = torch.full((rows, pitch), 0x7F, dtype=torch.uint8, device="cuda")
    shape = mfsdp.fp8_scale_shape(rows, cols, groups)
    scales = torch.full(shape, 255, dtype=torch.uint8, device="cuda")
    return mfsdp.Fp8Matrix(data.view(F8[kind])[:, :cols], scales, groups)


def _names(groups):
    return ("row", "col", "tile")[groups]


def _kind(m):
    return "e4m3" if m.data.dtype == torch.float8_e4m3fn else "e5m2"


def _held(m):
    return o8.values(_np(m.data), _np(m.scales), _names(m.groups))


def _check8(m, ref, tol):
    """m holds ref's values, which were known within tol, rounded once."""
    groups, kind = _names(m.groups), _kind(m)
    got = _held(m)
    bits, least, _ = o8.TYPES[kind]
    s = _np(m.scales)
    step = np.exp2(o8.spread(s, *ref.shape, groups) - 127.0 + least - bits)
    half = 2.0 ** -(bits + 1)
    bound = tol + np.maximum(half * (np.abs(ref) + tol), step / 2)
    assert (np.abs(got - ref) <= bound * (1 + 1e-12)).all(), float((np.abs(got - ref) / bound).max())
    lo = o8.quantize(np.maximum(np.abs(ref) - tol, 0), groups, kind)[1]
    hi = o8.quantize(np.abs(ref) + tol, groups, kind)[1]
    assert ((lo <= s) & (s <= hi)).all()


def _check(t, ref, tol):
    if t.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    err = np.abs(_np(t) - ref)
    assert (err <= tol + 1e-38).all(), float((err / (tol + 1e-38)).max())


def _mat(gen, rows, cols, dtype, std=1.0, mean=0.0, pitch=0, offset=0):
    base = torch.randn(rows * (cols + pitch) + offset, generator=gen, device="cuda") * std + mean
    return base.to(TYPES[dtype])[offset:].view(rows, cols + pitch)[:, :cols]


def _norm(rows, cols, dtype="bf16", params="f32", layer=True, kind="e4m3", residual=True, affine=True,
          with_y=True, dres=True, seed=0, pitch=0, offset=0, h8_kind="e4m3"):
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(seed)
    at = dict(pitch=pitch, offset=offset)
    x = _mat(gen, rows, cols, dtype, 0.5, **at)
    r = _mat(gen, rows, cols, dtype, 2.0, 0.5, **at) if residual else None
    w = (torch.randn(cols, generator=gen, device="cuda") * 0.3 + 1).to(TYPES[params]) if affine else None
    b = (torch.randn(cols, generator=gen, device="cuda")).to(TYPES[params]) if affine and layer else None
    h, y = (_mat(gen, rows, cols, dtype, **at) for _ in range(2))
    y8, h8 = _empty8(rows, cols, kind, extra=1), _empty8(rows, cols, h8_kind)
    mean = torch.full((rows,), float("nan"), device="cuda") if layer else None
    rstd = torch.full((rows,), float("nan"), device="cuda")
    code = mfsdp.NORM_LAYER if layer else mfsdp.NORM_RMS
    mfsdp.mfsdp_norm_residual_forward(code, x, r, w, b, 1e-5, h, y if with_y else None, y8, h8, mean,
                                      rstd)
    H = _np(x) + (_np(r) if residual else 0.0)
    Y, mu, rs = onorm.forward(H, _np(w), _np(b), 1e-5, layer)
    aw, ab = np.abs(_np(w)) if affine else 1.0, np.abs(_np(b)) if b is not None else 0.0
    A = (np.abs(H) + np.abs(H).mean(1, keepdims=True)) * rs[:, None]
    tol = 66 * U * (A * aw + ab)
    _check(h, H, U * np.abs(H))
    if with_y:
        _check(y, Y, tol)
    _check8(y8, Y, tol)
    _check8(h8, H, U * np.abs(H))
    assert (np.abs(_np(rstd) - rs) <= 66 * U * rs * (1 + (A * A).mean(1))).all()
    # backward, from h and from its checkpoint
    dy, d2 = _mat(gen, rows, cols, dtype, 0.1, **at), _mat(gen, rows, cols, dtype, 0.1, **at)
    for kept in (h, h8):
        dx = _mat(gen, rows, cols, dtype, **at)
        dw = torch.full((cols,), float("nan"), dtype=TYPES[params], device="cuda")
        db = torch.full((cols,), float("nan"), dtype=TYPES[params], device="cuda") if layer else None
        mfsdp.mfsdp_norm_residual_backward(code, dy, d2 if dres else None, kept, w, mean, rstd, dx, dw,
                                           db)
        K = _held(kept) if kept is h8 else _np(kept)
        DY, MU = _np(dy), _np(mean) if layer else np.zeros(rows)
        DX, DW, DB = onorm.backward(DY, K, _np(w), MU, _np(rstd), layer)
        rr = _np(rstd)[:, None]
        A = (np.abs(K) + np.abs(MU)[:, None]) * rr
        G = np.abs(DY) * aw
        m = lambda v: v.mean(1, keepdims=True)  # noqa: E731
        tol = 66 * U * rr * (G + m(G) + A * m(G * A))
        if dres:
            DX = DX + _np(d2)
            tol = tol + 2 * U * np.abs(_np(d2))
        _check(dx, DX, tol)
        _check(dw, DW, (66 + rows) * U * (np.abs(DY) * A).sum(0))
        if layer:
            _check(db, DB, (66 + rows) * U * np.abs(DY).sum(0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (5, 100), (33, 256), (7, 500), (100, 768),
                                       (9, 1001), (70, 1024), (17, 1100), (400, 2048), (5, 2056),
                                       (330, 4096), (40, 5000), (160, 8192), (3, 8200), (4, 20001)])
def test_norm_residual(rows, cols, layer, dtype):
    _norm(rows, cols, dtype=dtype, layer=layer, params="f32" if layer else "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(residual=False), dict(affine=False), dict(with_y=False),
                                dict(dres=False), dict(kind="e5m2", h8_kind="e5m2"), dict(offset=1),
                                dict(pitch=3), dict(pitch=8, offset=8), dict(params="bf16")])
def test_norm_residual_forms(kw, dtype):
    for rows, cols in ((20, 640), (12, 1300), (6, 3000), (3, 9000)):
        _norm(rows, cols, dtype=dtype, **kw)
        _norm(rows, cols, dtype=dtype, layer=False, **kw)


@pytest.mark.parametrize("cols", [384, 4096, 9000])
def test_norm_residual_in_place(cols):
    """The residual stream updated in place, and gradients written over their inputs."""
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r, dy, d2 = (_mat(gen, 50, cols, "bf16") for _ in range(4))
    w = torch.ones(cols, device="cuda")
    rstd = torch.empty(50, device="cuda")

    def run(h, y, dx):
        a = [t.clone() for t in (x, r, dy, d2)]
        h, y = a[h] if h is not None else torch.empty_like(x), a[y] if y is not None else \
            torch.empty_like(x)
        y8 = _empty8(50, cols)
        mfsdp.mfsdp_norm_residual_forward(mfsdp.NORM_RMS, a[0], a[1], w, None, 1e-6, h, y, y8, None,
                                          None, rstd)
        h0 = h.clone()
        dx = h if dx == "h" else a[dx] if dx is not None else torch.empty_like(x)
        mfsdp.mfsdp_norm_residual_backward(mfsdp.NORM_RMS, a[2], a[3], h, w, None, rstd, dx)
        return h0, y, dx, y8.data.view(torch.uint8), y8.scales

    want = run(None, None, None)
    for how in ((1, None, 2), (0, 1, 3), (1, 0, "h")):
        assert all(torch.equal(a, b) for a, b in zip(run(*how), want))


def test_norm_residual_non_finite():
    """A NaN or infinite entry reaches its own row alone; the other rows' groups are untouched."""
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, r = _mat(gen, 40, 768, "bf16"), _mat(gen, 40, 768, "bf16")
    clean = _empty8(40, 768)
    mfsdp.mfsdp_norm_residual_forward(mfsdp.NORM_RMS, x, r, None, None, 1e-6, y8=clean)
    x[3, 5], x[7, 700] = float("nan"), float("inf")
    y8, h8 = _empty8(40, 768), _empty8(40, 768)
    mfsdp.mfsdp_norm_residual_forward(mfsdp.NORM_RMS, x, r, None, None, 1e-6, y8=y8, h8=h8)
    bad = _np(y8.data)
    assert np.isnan(bad[3]).all() and np.isnan(bad[7, 700])
    keep = [i for i in range(40) if i not in (3, 7)]
    assert torch.equal(y8.data.view(torch.uint8)[keep], clean.data.view(torch.uint8)[keep])
    held = _held(h8)                              # in the checkpoint each stays where it is
    assert np.argwhere(np.isnan(held)).tolist() == [[3, 5], [7, 700]]


# ------------------------------------------------------------------------------------ activations
def _p_and_t(a):
    with np.errstate(over="ignore"):
        p = 1 / (1 + np.exp(-a))
    return p, ((4 + 4 * np.abs(a)) * (1 - p) + 6) * 2.0 ** -23


def _act(kind, rows, cols, dtype="bf16", y_kind="e4m3", grad="e5m2", with_y=True, seed=0, pitch=0,
         offset=0, std=1.5, halves=False):
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(seed)
    at = dict(pitch=pitch, offset=offset)
    glu = kind == "swiglu"
    if halves:
        both = _mat(gen, rows, 2 * cols, dtype, std)
        gate, up = both[:, :cols], both[:, cols:] if glu else None
    else:
        gate = _mat(gen, rows, cols, dtype, std, **at)
        up = _mat(gen, rows, cols, dtype, **at) if glu else None
    code = mfsdp.ACT_SWIGLU if glu else mfsdp.ACT_GELU
    y = _mat(gen, rows, cols, dtype, **at) if with_y else None
    y8, g8, u8 = _empty8(rows, cols, y_kind, extra=1), _empty8(rows, cols), _empty8(rows, cols)
    mfsdp.mfsdp_activation_forward(code, gate, up, y, y8, g8, u8 if glu else None)
    G, Up = _np(gate), _np(up) if glu else 1.0

    def arg(g):
        return g if glu else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)

    ref = o8.activation(kind, G, Up)
    p, T = _p_and_t(arg(G))
    tol = np.abs(G * Up) * (p * (T + 4 * U) + 1e-37)
    if with_y:
        _check(y, ref, tol)
    _check8(y8, ref, tol)
    _check8(g8, G, 0.0)
    if glu:
        _check8(u8, Up, 0.0)
    dy = _mat(gen, rows, cols, dtype, 0.1, **at)
    DY = _np(dy)
    for kept in ((gate, up), (g8, u8 if glu else None)):
        dg, du = (_mat(gen, rows, cols, dtype, **at) for _ in range(2))
        g_row, u_row = _empty8(rows, cols, grad), _empty8(rows, cols, grad, extra=2)
        g_col, u_col = _empty8(rows, cols, grad, 1), _empty8(rows, cols, "e4m3", 1)
        if glu:
            mfsdp.mfsdp_activation_backward(code, dy, *kept, dg, du, g_row, u_row, g_col, u_col)
        else:
            mfsdp.mfsdp_activation_backward(code, dy, *kept, dgate=dg, dgate8=g_row, dgate8_col=g_col)
        Gk = _held(kept[0]) if kept[0] is g8 else G
        Uk = (_held(kept[1]) if kept[1] is u8 else Up) if glu else 1.0
        DG, DU = o8.activation_grads(kind, DY, Gk, Uk)
        p, T = _p_and_t(arg(Gk))
        T = T + 8 * U
        if glu:
            tg = np.abs(DY * Uk) * (p * (1 + np.abs(Gk)) * T + 1e-37 * (1 + np.abs(Gk)))
        else:
            slope = np.abs(Gk) * 1.6 * (1 + 0.14 * Gk ** 2)
            tg = np.abs(DY) * (p * (1 + slope) * T + 1e-37 * (1 + slope))
        outs = [(dg, DG, tg), (g_row, DG, tg), (g_col, DG, tg)]
        if glu:
            tu = np.abs(DY * Gk) * (p * T + 1e-37)
            outs += [(du, DU, tu), (u_row, DU, tu), (u_col, DU, tu)]
        for out, want, tol in outs:
            (_check if isinstance(out, torch.Tensor) else _check8)(out, want, tol)


@pytest.mark.parametrize("kind", ["swiglu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (128, 128), (130, 257), (300, 1001), (5, 700)])
def test_activation(kind, dtype, rows, cols):
    _act(kind, rows, cols, dtype)


@pytest.mark.parametrize("kind", ["swiglu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(with_y=False), dict(y_kind="e5m2", grad="e4m3"), dict(offset=1),
                                dict(pitch=3), dict(pitch=8, offset=8), dict(std=40.0),
                                dict(halves=True)])
def test_activation_forms(kind, dtype, kw):
    _act(kind, 150, 392, dtype, **kw)


def test_activation_far_values():
    """Far from zero both activations are 0 or their input, with finite gradients."""
    from matrix_optimizer_owner_gb300 import mfsdp
    g = torch.tensor([[1e4, 1e20, 3e38, -1e4, -1e20, -3e38, 0.0, float("nan")]], device="cuda")
    one = torch.ones_like(g)
    for code, up in ((mfsdp.ACT_SWIGLU, one), (mfsdp.ACT_GELU, None)):
        y, dg = torch.empty_like(g), torch.empty_like(g)
        mfsdp.mfsdp_activation_forward(code, g, up, y)
        mfsdp.mfsdp_activation_backward(code, one, g, up, dgate=dg)
        assert torch.equal(y[0, :7], torch.clamp(g[0, :7], min=0.0)) and y[0, 7].isnan()
        assert dg[0, :7].tolist() == [1, 1, 1, 0, 0, 0, 0.5] and dg[0, 7].isnan()
