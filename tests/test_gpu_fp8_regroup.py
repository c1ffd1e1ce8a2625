"""Regrouping at the top of the range.  fp32's largest values are 2^128 in 8 bits, which is no fp32 value:
regrouped, they stay 2^128, and the results are the float64 oracle's for what the source holds, bit for bit.
A magnitude above 2^128, which only scales made elsewhere give, becomes 2^128.  The activations' gradients
start from fp32's largest value there, and stay finite."""

import numpy as np
import pytest
import torch

from oracle import fp8 as oracle

pytestmark = pytest.mark.gpu
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
GROUPS = {"row": 0, "col": 1, "tile": 2}


def _np(t):
    return t.detach().double().cpu().numpy()


def _new(rows, cols, groups, kind):
    from matrix_optimizer_owner_gb300 import mfsdp
    return mfsdp.fp8_empty(rows, cols, GROUPS[groups], F8[kind])


def _same(m, want, groups, kind):
    q, s = oracle.quantize(want, groups, kind)
    assert np.array_equal(m.scales.view(torch.uint8).cpu().numpy(), s)
    assert np.array_equal(_np(m.data), q, equal_nan=True)


@pytest.mark.parametrize("rows,cols", [(8, 256), (130, 300), (256, 384)])
@pytest.mark.parametrize("src", ["row", "col", "tile"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_largest_values_survive(kind, src, rows, cols):
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    big = torch.finfo(torch.float32).max
    for i, (r, c) in enumerate([(0, 0), (3, 7), (3, 200), (rows - 1, cols - 1), (rows // 2, 130)]):
        x[r, c] = (big, -big, 0.97 * big, -0.99 * big, 0.6 * big)[i]
    x[5, 5] = float("inf")
    held = _new(rows, cols, src, kind)
    mfsdp.mfsdp_quantize_fp8(x, held)
    want = oracle.values(*oracle.quantize(_np(x), src, kind), src)
    assert (np.abs(want) == 2.0 ** 128).sum() >= 3 and np.isnan(want).sum() == 1
    for groups in ("row", "col", "tile"):
        for to in ("e4m3", "e5m2"):
            out = _new(rows, cols, groups, to)
            mfsdp.mfsdp_regroup_fp8(held, out)
            _same(out, want, groups, to)
    a, b = _new(rows, cols, "row", "e5m2"), _new(rows, cols, "col", kind)
    mfsdp.mfsdp_regroup_fp8(held, a, b)
    _same(a, want, "row", "e5m2")
    _same(b, want, "col", kind)


@pytest.mark.parametrize("src", ["row", "col", "tile"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("scale", [238, 239, 240, 246, 247, 248, 254])
def test_every_code_of_large_scales(kind, src, scale):
    """Every finite value under a scale near the end of its range."""
    from matrix_optimizer_owner_gb300 import mfsdp
    rows, cols = 256, 256
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(rows, 1)
    codes = torch.where(codes.view(F8[kind]).float().isfinite(), codes, 0)
    m = _new(rows, cols, src, kind)
    m.data.copy_(codes.view(F8[kind]))
    m.scales.view(torch.uint8).fill_(scale)
    held = oracle.values(_np(m.data), m.scales.view(torch.uint8).cpu().numpy(), src)
    held = np.clip(held, -2.0 ** 128, 2.0 ** 128)
    for groups in ("row", "col", "tile"):
        for to in ("e4m3", "e5m2"):
            out = _new(rows, cols, groups, to)
            mfsdp.mfsdp_regroup_fp8(m, out)
            _same(out, held, groups, to)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activation_gradients_at_the_largest_values(dtype):
    """Where a gate is far from zero the activation passes it or nothing: dgate is dy up or 0 for SwiGLU, dy
    or 0 for GELU, dup is dy gate or 0."""
    from matrix_optimizer_owner_gb300 import mfsdp
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    big = torch.finfo(t).max
    gate = torch.tensor([[big, -big, 0.98 * big, 0.0]] * 2, device="cuda").to(t)
    up, dy = torch.full_like(gate, 0.5), torch.full_like(gate, 0.25)
    g8, u8 = _new(2, 4, "row", "e4m3"), _new(2, 4, "row", "e4m3")
    mfsdp.mfsdp_activation_forward(mfsdp.ACT_SWIGLU, gate, up, torch.empty_like(gate), gate8=g8, up8=u8)
    assert np.array_equal(_np(g8.data)[0], [256, -256, 256, 0])
    dg, du = torch.empty_like(dy), torch.empty_like(dy)
    mfsdp.mfsdp_activation_backward(mfsdp.ACT_SWIGLU, dy, g8, u8, dg, du)
    most = float(torch.tensor(torch.finfo(torch.float32).max / 4).to(t))       # (rounded to bf16: 2^126)
    assert dg[0].tolist() == [0.125, 0, 0.125, 0.0625] and du[0].tolist() == [most, 0, most, 0]
    mfsdp.mfsdp_activation_backward(mfsdp.ACT_GELU, dy, g8, None, dgate=dg)
    assert dg[0].tolist() == [0.25, 0, 0.25, 0.125]
