"""Backward passes whose blocks take several tiles or rows in turn: the rings of copied-ahead inputs wrap, the
scales carried along, the shared memory of the column scales and the column sums are used again.

Against the formulas in float64, computed on the device (its 8-bit rounding is pinned to the oracle's here).
Bounds are those of the norms and activations (u = 2^-24):
    |ddx| <= 66 u rstd (|g| + mean|g| + A mean(|g| A)) + 2 u |dres|,  A = (|h| + |mean|) rstd;
    dgate and dup within T + 8 u of the products they are made of, T = ((4 + 4 |a|) (1 - p) + 6) 2^-23.
A column's sum over R rows takes at most R / (S W) additions in a register (S the SMs, each with a block at
least, W the rows that a block holds: 8 of up to 1024 entries, else 1), 8 over a block's warps, and 8 S / 32 + 32 over
the blocks (8 S at most): within (66 + R / (S W) + 8 + 8 S / 32 + 33) u of its sum of absolute values, which a
row that is left out, a share of about 1 / R, is not.
"""

import numpy as np
import pytest
import torch

from oracle import fp8 as oracle

U = 2.0 ** -24
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TOP = {"e4m3": 9, "e5m2": 16}                     # the largest value is 7/8 2^TOP
ROW, COL = 0, 1


# ------------------------------------------------------------------------------------ 8 bits in float64
def _spread(s, groups, shape):
    s = s.repeat_interleave(128, 1)[:, :shape[1]] if groups == ROW else s
    return s if groups == ROW else s.repeat_interleave(128, 0)[:shape[0]]


def _scales(x, groups, kind):
    """The groups' scale bytes of finite values."""
    rows, cols = x.shape
    a = x.abs() if groups == ROW else x.abs().T
    a = torch.nn.functional.pad(a, (0, -a.shape[1] % 128)).unflatten(1, (-1, 128)).amax(2)
    frac, e = torch.frexp(a)
    s = torch.where(a > 0, (127 - TOP[kind] + e + (frac > 0.875)).clamp_(min=0), 0)
    return s if groups == ROW else s.T


def _held(m):
    s = m.scales.view(torch.uint8).double()
    return m.data.double() * torch.exp2(_spread(s, m.groups, m.data.shape) - 127)


def _kind(m):
    return "e4m3" if m.data.dtype == torch.float8_e4m3fn else "e5m2"


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_scales_are_the_oracles(kind):
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(300, 257, generator=gen, dtype=torch.float64)
    x *= torch.exp2(torch.randint(-140, 60, x.shape, generator=gen).double())
    x[:, :128] *= torch.exp2(torch.randint(-140, 1, (300, 1), generator=gen).double())
    big = oracle.TYPES[kind][2]
    x[3, 128:256] = 0
    x[4, 128:256], x[5, 128:256] = big, big * (1 + 2.0 ** -50)
    for groups, name in ((ROW, "row"), (COL, "col")):
        assert np.array_equal(_scales(x, groups, kind).numpy(), oracle.quantize(x.numpy(), name, kind)[1])


def _check8(m, ref, tol):
    """m holds ref's values, which were known within tol, rounded once; NaN where ref is not finite."""
    bits, least, _ = oracle.TYPES[_kind(m)]
    got, bad = _held(m), ~ref.isfinite()
    assert torch.equal(got.isnan(), bad)
    got, ref, tol = (torch.where(bad, 0.0, t) for t in (got, ref, tol))
    s = m.scales.view(torch.uint8)
    step = torch.exp2(_spread(s.double(), m.groups, ref.shape) - 127 + least - bits)
    bound = tol + torch.maximum(2.0 ** -(bits + 1) * (ref.abs() + tol), step / 2)
    err = (got - ref).abs()
    assert (err <= bound * (1 + 1e-12)).all(), float((err / bound).max())
    lo = _scales((ref.abs() - tol).clamp(min=0), m.groups, _kind(m))
    hi = _scales(ref.abs() + tol, m.groups, _kind(m))
    assert ((lo <= s) & (s <= hi)).all()


def _check(t, ref, tol):
    bad = ~ref.isfinite()
    assert not t[bad].isfinite().any()
    if t.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err, tol = (t.double() - ref).abs()[~bad], tol[~bad] + 1e-38
    assert (err <= tol).all(), float((err / tol).max())


def _mat(gen, rows, cols, dtype, std=1.0, mean=0.0):
    return (torch.randn(rows, cols, generator=gen, device="cuda") * std + mean).to(TYPES[dtype])


# ------------------------------------------------------------------------------------ activations
def _gate(kind, g):
    a = g if kind == "swiglu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    p = 1 / (1 + torch.exp(-a))
    return p, ((4 + 4 * a.abs()) * (1 - p) + 6) * 2.0 ** -23 + 8 * U


@pytest.mark.gpu
@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("kind,dtype,rows,cols", [
    ("swiglu", "bf16", 1500, 6104), ("gelu", "bf16", 1500, 6104), ("swiglu", "bf16", 1500, 6101),
    ("swiglu", "f32", 1280, 6144), ("gelu", "f32", 1500, 6104), ("gelu", "f32", 1300, 5003)])
def test_activation_gradients_of_several_tiles_a_block(kind, dtype, rows, cols, checkpoint):
    """All results of both groupings; entries that are not finite make every third tile row look at its
    columns twice."""
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    glu = kind == "swiglu"
    gate, up = _mat(gen, rows, cols, dtype, 1.5), _mat(gen, rows, cols, dtype) if glu else None
    dy = _mat(gen, rows, cols, dtype, 0.1)
    dy *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=gen, device="cuda")).to(dy.dtype)
    at = torch.arange(10, rows, 384, device="cuda")
    dy[at[:, None], torch.arange(7, cols, 300, device="cuda")] = float("inf")
    dy[at[:, None] + 1, torch.arange(5, cols, 1000, device="cuda")] = float("nan")
    new = lambda groups, k: mfsdp.fp8_empty(rows, cols, groups, F8[k])  # noqa: E731
    if checkpoint:
        kept = [None if t is None else new(ROW, "e4m3") for t in (gate, up)]
        for t, m in zip((gate, up), kept):
            if m is not None:
                mfsdp.mfsdp_quantize_fp8(t, m)
        G, V = _held(kept[0]), _held(kept[1]) if glu else 1.0
    else:
        kept, G, V = (gate, up), gate.double(), up.double() if glu else 1.0
    dg, du = torch.empty_like(dy), torch.empty_like(dy) if glu else None
    g_row, g_col = new(ROW, "e5m2"), new(COL, "e4m3")
    u_row, u_col = (new(ROW, "e4m3"), new(COL, "e5m2")) if glu else (None, None)
    code = mfsdp.ACT_SWIGLU if glu else mfsdp.ACT_GELU
    mfsdp.mfsdp_activation_backward(code, dy, *kept, dg, du, g_row, u_row, g_col, u_col)
    D = dy.double()
    p, T = _gate(kind, G)
    if glu:
        DG, DU = D * V * p * (1 + G * (1 - p)), D * G * p
        tg = (D * V).abs() * (p * (1 + G.abs()) * T + 1e-37 * (1 + G.abs()))
        tu = (D * G).abs() * (p * T + 1e-37)
    else:
        slope = 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * G ** 2)
        DG, DU = D * (p + G * p * (1 - p) * slope), None
        s = G.abs() * 1.6 * (1 + 0.14 * G ** 2)
        tg = D.abs() * (p * (1 + s) * T + 1e-37 * (1 + s))
    DG = torch.where(D.isfinite(), DG, float("nan"))
    _check(dg, DG, tg)
    _check8(g_row, DG, tg)
    _check8(g_col, DG, tg)
    if glu:
        DU = torch.where(D.isfinite(), DU, float("nan"))
        _check(du, DU, tu)
        _check8(u_row, DU, tu)
        _check8(u_col, DU, tu)


# ------------------------------------------------------------------------------------ norms
@pytest.mark.gpu
@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("dtype,rows,cols", [
    ("bf16", 9001, 768), ("bf16", 9001, 500), ("bf16", 20003, 256), ("bf16", 9003, 1024),
    ("bf16", 4001, 2048), ("bf16", 3001, 4096), ("bf16", 1501, 8192), ("bf16", 3003, 3001),
    ("f32", 9001, 768), ("f32", 3001, 2000), ("f32", 2001, 4096), ("f32", 1501, 6000),
    ("bf16", 501, 8200)])
def test_norm_gradients_of_several_rows_a_block(dtype, rows, cols, layer, checkpoint):
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x, r = _mat(gen, rows, cols, dtype, 0.5), _mat(gen, rows, cols, dtype, 2.0, 0.5)
    w = torch.randn(cols, generator=gen, device="cuda") * 0.3 + 1
    b = torch.randn(cols, generator=gen, device="cuda") if layer else None
    h, y = torch.empty_like(x), torch.empty_like(x)
    h8 = mfsdp.fp8_empty(rows, cols, ROW)
    mean, rstd = torch.empty(rows, device="cuda") if layer else None, torch.empty(rows, device="cuda")
    code = mfsdp.NORM_LAYER if layer else mfsdp.NORM_RMS
    mfsdp.mfsdp_norm_residual_forward(code, x, r, w, b, 1e-5, h, y, None, h8, mean, rstd)
    dy, d2 = _mat(gen, rows, cols, dtype, 0.1), _mat(gen, rows, cols, dtype, 0.1)
    dx, dw = torch.empty_like(dy), torch.full_like(w, float("nan"))
    db = torch.full_like(w, float("nan")) if layer else None
    mfsdp.mfsdp_norm_residual_backward(code, dy, d2, h8 if checkpoint else h, w, mean, rstd, dx, dw, db)
    K, D, W = _held(h8) if checkpoint else h.double(), dy.double(), w.double()
    mu, rs = mean.double()[:, None] if layer else 0.0, rstd.double()[:, None]
    z, g = (K - mu) * rs, D * W
    m = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    A = (K.abs() + abs(mu)) * rs
    ref = rs * (g - (m(g) if layer else 0.0) - z * m(g * z)) + d2.double()
    tol = 66 * U * rs * (g.abs() + m(g.abs()) + A * m(g.abs() * A)) + 2 * U * d2.double().abs()
    _check(dx, ref, tol)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    many = 66 + rows / (sms * (8 if cols <= 1024 else 1)) + 8 + 8 * sms / 32 + 33
    _check(dw, (D * z).sum(0), many * U * (D.abs() * A).sum(0))
    if layer:
        _check(db, D.sum(0), many * U * D.abs().sum(0))
