"""8-bit matrices (quantize, regroup, dequantize) and their products against the float64 oracle.

A scaled value is exact and its rounding is defined, so 8-bit results are equal to the oracle's.

A product's entry is a sum of K exact products, S = sum |a b|: the tensor cores add them 32 at a time
into fp32 without rounding to nearest, so |dc| <= (K / 32 + 8) 2^-22 S, and sums outside them (chunks
and slices of the contraction, what C held) add at most (K / 1024 + 34) 2^-24 (S + |c|); a result in
bf16 is rounded once (2^-9 of a power of two: 2^-8 of the value).
"""

import numpy as np
import pytest
import torch

from oracle import fp8 as oracle

pytestmark = pytest.mark.gpu
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GROUPS = {"row": 0, "col": 1, "tile": 2}


def _np(t):
    return t.detach().double().cpu().numpy()


def _empty8(rows, cols, groups, kind, extra=0, fill=0xA5):
    """An 8-bit matrix inside a larger buffer (a pitch of `extra` more vectors), all bytes `fill`."""
    from matrix_optimizer_owner_gb300 import mfsdp
    pitch = -(-cols // 16) * 16 + 16 * extra
    data = torch.full((rows, pitch), fill, dtype=torch.uint8, device="cuda")
    gr, gc = oracle.scale_shape(rows, cols, groups)
    scales = torch.full((gr, gc + extra), fill, dtype=torch.uint8, device="cuda")
    m = mfsdp.Fp8Matrix(data.view(F8[kind])[:, :cols], scales[:, :gc], GROUPS[groups])
    return m, data, scales


def _check8(m, data, scales, x, groups, kind):
    rows, cols = x.shape
    q, s = oracle.quantize(x, groups, kind)
    gr, gc = s.shape
    assert np.array_equal(scales.cpu().numpy()[:, :gc], s)
    got = _np(m.data)
    assert np.array_equal(np.isnan(got), np.isnan(q))
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(q))
    assert (data[:, cols:] == 0xA5).all() and (scales[:, gc:] == 0xA5).all()


def _wide(rows, cols, dtype, seed=0, offset=0, pitch=0):
    """Values of very different sizes, zeros, subnormals and whole zero groups among them."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = rows * (cols + pitch) + offset
    v = torch.randn(n, generator=gen, device="cuda")
    v *= torch.exp2(torch.randint(-20, 20, (n,), generator=gen, device="cuda").float())
    v[torch.rand(n, generator=gen, device="cuda") < 0.05] = 0
    x = v.to(TYPES[dtype])[offset:].view(rows, cols + pitch)[:, :cols]
    if rows > 4 and cols > 300:
        x[2, 128:256] = 0
        x[3, :128] = 1e-39
        x[4, :128] *= 1e25 if dtype == "f32" else 1e20
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols,offset,pitch", [
    (1, 1, 0, 0), (1, 4096, 0, 0), (3, 130, 0, 6), (129, 257, 0, 7), (128, 128, 0, 0),
    (200, 384, 1, 1), (257, 1001, 0, 0), (5, 2000, 3, 0)])
def test_quantize(dtype, kind, rows, cols, offset, pitch):
    from matrix_optimizer_owner_gb300 import mfsdp
    x = _wide(rows, cols, dtype, rows + cols, offset, pitch)
    ref = _np(x)
    for groups in ("row", "col", "tile"):
        out = _empty8(rows, cols, groups, kind, extra=1)
        mfsdp.mfsdp_quantize_fp8(x, out[0])
        _check8(*out, ref, groups, kind)
    a, b = _empty8(rows, cols, "row", kind), _empty8(rows, cols, "col", kind, extra=2)
    mfsdp.mfsdp_quantize_fp8(x, a[0], b[0])
    _check8(*a, ref, "row", kind)
    _check8(*b, ref, "col", kind)
    a, b = _empty8(rows, cols, "row", "e5m2"), _empty8(rows, cols, "col", kind)
    mfsdp.mfsdp_quantize_fp8(x, b[0], a[0])                 # the other way round, types apart
    _check8(*a, ref, "row", "e5m2")
    _check8(*b, ref, "col", kind)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_quantize_borders(kind):
    """Largest values at and beside the border of a scale, ties, and values that are not finite."""
    from matrix_optimizer_owner_gb300 import mfsdp
    big = oracle.TYPES[kind][2]
    x = torch.zeros(8, 256, device="cuda")
    x[0, 0] = big                                            # just fits
    x[1, 0] = float(np.nextafter(np.float32(big), np.float32(np.inf)))
    x[2, 0] = float(np.nextafter(np.float32(big), np.float32(0)))
    x[3, :] = torch.arange(256, device="cuda") / 16 + 1 / 32  # ties among them
    x[3, 255] = -big
    x[4, 3], x[4, 130], x[4, 131] = float("inf"), float("nan"), float("-inf")
    x[4, 4], x[4, 140] = 3.0, -5.5
    x[5, :] = float("inf")                                    # nothing finite
    x[6, 0], x[6, 200] = torch.finfo(torch.float32).max, -torch.finfo(torch.float32).max
    x[7, 0], x[7, 1] = 2.0 ** -149, 2.0 ** -126
    for groups in ("row", "col", "tile"):
        out = _empty8(8, 256, groups, kind)
        mfsdp.mfsdp_quantize_fp8(x, out[0])
        _check8(*out, _np(x), groups, kind)
        back = torch.empty(8, 256, device="cuda")
        mfsdp.mfsdp_dequantize_fp8(out[0], back)
        q, s = oracle.quantize(_np(x), groups, kind)
        # fp32's largest value is 2^128 (1 - 2^-24): in 8 bits it is 2^128, which fp32 has as infinity
        with np.errstate(over="ignore"):
            want = oracle.values(q, s, groups).astype(np.float32).astype(np.float64)
        assert np.array_equal(_np(back), want, equal_nan=True)


@pytest.mark.parametrize("rows,cols", [(1, 7), (130, 300), (300, 1001), (256, 512)])
@pytest.mark.parametrize("src", ["row", "col", "tile"])
def test_regroup_and_dequantize(rows, cols, src):
    from matrix_optimizer_owner_gb300 import mfsdp
    x = _wide(rows, cols, "bf16", 3)
    m = _empty8(rows, cols, src, "e4m3")[0]
    mfsdp.mfsdp_quantize_fp8(x, m)
    held = oracle.values(*oracle.quantize(_np(x), src, "e4m3"), src)
    for dtype in ("f32", "bf16"):
        base = torch.full((rows, cols + 3), 7.0, dtype=TYPES[dtype], device="cuda")
        mfsdp.mfsdp_dequantize_fp8(m, base[:, :cols])
        # exact, but for what bf16 and fp32 hold as subnormals (none here)
        assert np.array_equal(_np(base[:, :cols]), held) and (base[:, cols:] == 7).all()
    for groups, kind in (("row", "e4m3"), ("col", "e4m3"), ("tile", "e5m2")):
        out = _empty8(rows, cols, groups, kind, extra=1)
        mfsdp.mfsdp_regroup_fp8(m, out[0])
        _check8(*out, held, groups, kind)
    a, b = _empty8(rows, cols, "row", "e5m2"), _empty8(rows, cols, "col", "e4m3")
    mfsdp.mfsdp_regroup_fp8(m, a[0], b[0])
    _check8(*a, held, "row", "e5m2")
    _check8(*b, held, "col", "e4m3")


def test_scale_255_is_nan():
    from matrix_optimizer_owner_gb300 import mfsdp
    m, _, scales = _empty8(4, 256, "row", "e4m3", fill=0)
    scales[1, 1] = 255
    out = torch.empty(4, 256, device="cuda")
    mfsdp.mfsdp_dequantize_fp8(m, out)
    assert out[1, 128:].isnan().all() and int(out.isnan().sum()) == 128


# ------------------------------------------------------------------------------------ products
def _operand(rows, cols, groups, kind, gen, extra=0, spread=3):
    """A random 8-bit matrix: any finite code, scales a few binades apart."""
    m, data, scales = _empty8(rows, cols, groups, kind, extra)
    codes = torch.randint(256, data.shape, generator=gen, device="cuda").to(torch.uint8)
    top = 0x78 if kind == "e4m3" else 0x5C                   # up to 240 and 240
    codes = torch.where((codes & 0x7F) > top, codes & 0x8F, codes)
    data.copy_(codes)                                        # the padding holds values too
    scales.copy_(torch.randint(127 - spread, 127 + spread + 1, scales.shape, generator=gen,
                               device="cuda").to(torch.uint8))
    want = oracle.values(_np(m.data), _np(m.scales), groups)
    return m, want


def _product(m, n, k, trans_a, trans_b, dtype, kinds=("e4m3", "e4m3"), groups=None, accumulate=False,
             seed=0, extra=0, offset=0, pitch=0):
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ga = (groups or ("", ""))[0] or ("col" if trans_a else "row")
    gb = (groups or ("", ""))[1] or ("row" if trans_b else "col")
    a, va = _operand(*((k, m) if trans_a else (m, k)), ga, kinds[0], gen, extra)
    b, vb = _operand(*((n, k) if trans_b else (k, n)), gb, kinds[1], gen, extra)
    base = torch.randn(m * (n + pitch) + offset, generator=gen, device="cuda").to(TYPES[dtype])
    c = base[offset:].view(m, n + pitch)[:, :n]
    old, keep = _np(c).copy(), base[offset:].view(m, n + pitch)[:, n:].clone()
    mfsdp.mfsdp_gemm_fp8(a, b, c, trans_a=trans_a, trans_b=trans_b, accumulate=accumulate)
    A, B = va.T if trans_a else va, vb if not trans_b else vb.T
    ref, S = A @ B, np.abs(A) @ np.abs(B)
    if accumulate:
        ref = ref + old
    tol = (k / 32 + 8) * 2.0 ** -22 * S + (k / 1024 + 34) * 2.0 ** -24 * (S + np.abs(ref)) + 1e-30
    if dtype == "bf16":
        tol = tol + np.abs(ref) * 2.0 ** -8
    err = np.abs(_np(c) - ref)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:5])
    assert torch.equal(base[offset:].view(m, n + pitch)[:, n:], keep)
    return a, b, c


@pytest.mark.parametrize("m,n,k", [(1400, 1500, 10253), (1280, 1030, 9000), (700, 2500, 12288)])
def test_gemm_few_tiles_long_contraction(m, n, k):
    """Two halves of the contraction at a time, joined at the end."""
    _product(m, n, k, True, False, "f32")
    _product(m, n, k, False, True, "bf16", pitch=1)
    _product(m, n, k, True, False, "bf16", accumulate=True, kinds=("e5m2", "e4m3"))


ORIENT = [(False, True), (False, False), (True, False), (True, True)]


@pytest.mark.parametrize("trans_a,trans_b", ORIENT)
@pytest.mark.parametrize("m,n,k", [(256, 256, 128), (512, 256, 1024), (257, 300, 130),
                                   (300, 513, 700), (129, 1000, 1), (1000, 140, 2049),
                                   (70, 300, 900), (1500, 2300, 384), (260, 300, 20000)])
def test_gemm(m, n, k, trans_a, trans_b):
    _product(m, n, k, trans_a, trans_b, "f32", extra=1)
    _product(m, n, k, trans_a, trans_b, "bf16")


@pytest.mark.parametrize("trans_a,trans_b", ORIENT)
@pytest.mark.parametrize("m,n,k", [(1, 128, 128), (1, 1000, 4096), (3, 257, 513), (16, 64, 32),
                                   (17, 2048, 1000), (33, 300, 2048), (64, 129, 700), (128, 1000, 4000),
                                   (100, 1, 300), (1, 1, 1), (2, 20000, 128), (500, 40, 1500)])
def test_gemm_narrow(m, n, k, trans_a, trans_b):
    _product(m, n, k, trans_a, trans_b, "f32", extra=1)
    _product(m, n, k, trans_a, trans_b, "bf16")


@pytest.mark.parametrize("m,n", [(300, 400), (5, 300), (300, 5)])
@pytest.mark.parametrize("kinds", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_gemm_types(m, n, kinds):
    for t in ORIENT:
        _product(m, n, 500, *t, "f32", kinds=kinds)


@pytest.mark.parametrize("m,n", [(300, 400), (5, 400), (400, 5)])
def test_gemm_tile_scales(m, n):
    for t in ORIENT:
        _product(m, n, 900, *t, "f32", groups=("tile", ""))
        _product(m, n, 900, *t, "f32", groups=("", "tile"))
        _product(m, n, 900, *t, "bf16", groups=("tile", "tile"))


@pytest.mark.parametrize("m,n,k", [(300, 400, 700), (4, 400, 700), (300, 3, 700), (300, 260, 9000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gemm_accumulate_and_strides(m, n, k, dtype):
    for kw in (dict(), dict(offset=1), dict(pitch=3), dict(pitch=8), dict(offset=2, pitch=5)):
        _product(m, n, k, False, True, dtype, accumulate=True, **kw)
        _product(m, n, k, True, False, dtype, accumulate=False, **kw)


def test_gemm_empty():
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(0)
    a, _ = _operand(0, 256, "col", "e4m3", gen)
    b, _ = _operand(0, 300, "col", "e4m3", gen)
    c = torch.ones(256, 300, device="cuda")
    mfsdp.mfsdp_gemm_fp8(a, b, c, trans_a=True, accumulate=True)
    assert (c == 1).all()
    mfsdp.mfsdp_gemm_fp8(a, b, c, trans_a=True)              # no tokens: a zero gradient
    assert (c == 0).all()
    x, _ = _operand(0, 256, "row", "e4m3", gen)
    w, _ = _operand(300, 256, "tile", "e4m3", gen)
    mfsdp.mfsdp_gemm_fp8(x, w, torch.empty(0, 300, device="cuda"), trans_b=True)


@pytest.mark.parametrize("m,n", [(300, 400), (3, 400)])
def test_gemm_nan_stays_in_its_row(m, n):
    """A NaN value or scale of A's row reaches that row of C and no other."""
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(5)
    a, va = _operand(m, 640, "row", "e4m3", gen)
    b, vb = _operand(n, 640, "row", "e4m3", gen)
    a.data.view(torch.uint8)[1, 300] = 0x7F
    a.scales[2, 4] = 255
    c = torch.empty(m, n, device="cuda")
    mfsdp.mfsdp_gemm_fp8(a, b, c, trans_b=True)
    bad = c.isnan().any(1).cpu().numpy()
    assert c[1].isnan().all() and c[2].isnan().all() and bad.sum() == 2


def test_gemm_repeats_and_streams():
    """The same bits each time, on another stream too."""
    from matrix_optimizer_owner_gb300 import mfsdp
    for m, n, k in ((300, 260, 20000), (600, 700, 512), (7, 900, 4096)):
        a, b, c = _product(m, n, k, True, False, "f32")
        first = c.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for kw in (dict(), dict(stream=s)):
            c.zero_()
            s.wait_stream(torch.cuda.current_stream())
            mfsdp.mfsdp_gemm_fp8(a, b, c, trans_a=True, **kw)
            torch.cuda.synchronize()
            assert torch.equal(c, first)
    assert mfsdp.mfsdp_query_status() == 0
