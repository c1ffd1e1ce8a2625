"""The 8-bit operators without a GPU: refusals before any launch (pointers here are made-up addresses that
no kernel ever sees), the binding's checks, and the float64 oracle against torch's float8 casts and
automatic differentiation."""

import ctypes as C
import os

import numpy as np
import pytest
import torch

from oracle import fp8 as oracle

P = 4096          # an address with every alignment
EINVAL, ESHAPE, EALIGN, EWORKSPACE = -1, -2, -3, -5
ROW, COL, TILE = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from matrix_optimizer_owner_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from matrix_optimizer_owner_gb300 import build
        build.build()
    return _lib.load()


def _m(data=P, ld=256, scales=P, ld_s=256, dtype=0, groups=ROW):
    from matrix_optimizer_owner_gb300._lib import Fp8Struct
    return Fp8Struct(data, ld, scales, ld_s, dtype, groups)


def _call(fn, good, **changes):
    args = dict(good, **changes)
    assert set(args) == set(good)
    return fn(*args.values())


BAD = [(dict(dtype=2), EINVAL), (dict(groups=3), EINVAL), (dict(groups=-1), EINVAL),
       (dict(data=None), EINVAL), (dict(scales=None), EINVAL), (dict(ld=192), EINVAL),
       (dict(ld_s=1), EINVAL), (dict(data=P + 8), EALIGN), (dict(ld=264), EALIGN)]


@pytest.mark.parametrize("change,status", BAD)
def test_matrix_refusals(lib, change, status):
    """A malformed 8-bit matrix is refused wherever one is taken (200 x 200 here)."""
    bad, good = _m(**change), _m()
    if change.get("groups", ROW) == ROW:       # what takes ROW matrices alone
        assert lib.mfsdp_norm_residual_forward(0, 200, 200, 1, 0, P, 256, None, 0, P, P, 1e-5, None, 0,
                                               None, 0, bad, None, P, P, None) == status
        assert lib.mfsdp_norm_residual_forward(0, 200, 200, 1, 0, P, 256, None, 0, P, P, 1e-5, None, 0,
                                               P, 256, None, bad, P, P, None) == status
        assert lib.mfsdp_norm_residual_backward(0, 200, 200, 1, 0, P, 256, None, 0, None, 0, bad, P, P,
                                                P, P, 256, P, P, P, 1 << 24, None) == status
        assert lib.mfsdp_activation_forward(0, 200, 200, 1, P, 256, P, 256, None, 0, bad, None, None,
                                            None) == status
        assert lib.mfsdp_activation_backward(0, 200, 200, 1, P, 256, None, 0, bad, None, 0, good, P, 256,
                                             P, 256, None, None, None, None, None) == status
    assert lib.mfsdp_quantize_fp8(200, 200, 1, P, 256, bad, None, None) == status
    assert lib.mfsdp_regroup_fp8(200, 200, bad, good, None, None) == status
    assert lib.mfsdp_regroup_fp8(200, 200, good, bad, None, None) == status
    assert lib.mfsdp_dequantize_fp8(200, 200, bad, 0, P, 256, None) == status
    assert lib.mfsdp_gemm_fp8(200, 200, 200, bad, 0, good, 1, 0, 0, P, 256, None) == status
    assert lib.mfsdp_gemm_fp8(200, 200, 200, good, 0, bad, 1, 0, 0, P, 256, None) == status


QUANT = dict(rows=8, cols=200, dtype=1, x=P, ld=200, out=None, also=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), ESHAPE), (dict(cols=0), ESHAPE), (dict(rows=1 << 31), ESHAPE),
    (dict(cols=1 << 31), ESHAPE), (dict(dtype=2), EINVAL), (dict(x=None), EINVAL),
    (dict(ld=199), EINVAL), (dict(x=P + 1), EALIGN), (dict(out=None), EINVAL),
    (dict(also=ROW), EINVAL), (dict(also=TILE), EINVAL), (dict(rows=0, x=None), 0)])
def test_quantize_refusals(lib, change, status):
    change = dict(change)
    out = change.pop("out", ROW)
    also = change.pop("also", None)
    assert _call(lib.mfsdp_quantize_fp8, QUANT, **change, out=None if out is None else _m(groups=out),
                 also=None if also is None else _m(groups=also)) == status


def test_regroup_and_dequantize_refusals(lib):
    good = _m()
    assert lib.mfsdp_regroup_fp8(8, 200, None, good, None, None) == EINVAL
    assert lib.mfsdp_regroup_fp8(8, 200, good, None, None, None) == EINVAL
    assert lib.mfsdp_regroup_fp8(8, 200, good, _m(groups=TILE), _m(groups=COL), None) == EINVAL
    assert lib.mfsdp_regroup_fp8(8, 0, good, good, None, None) == ESHAPE
    assert lib.mfsdp_regroup_fp8(0, 200, good, good, None, None) == 0
    assert lib.mfsdp_dequantize_fp8(8, 200, None, 0, P, 200, None) == EINVAL
    assert lib.mfsdp_dequantize_fp8(8, 200, good, 2, P, 200, None) == EINVAL
    assert lib.mfsdp_dequantize_fp8(8, 200, good, 0, None, 200, None) == EINVAL
    assert lib.mfsdp_dequantize_fp8(8, 200, good, 0, P, 199, None) == EINVAL
    assert lib.mfsdp_dequantize_fp8(8, 200, good, 0, P + 2, 200, None) == EALIGN
    assert lib.mfsdp_dequantize_fp8(0, 200, good, 0, None, 200, None) == 0


GEMM = dict(m=100, n=200, k=150, a=None, ta=0, b=None, tb=1, acc=0, dtype=0, c=P, ld_c=200, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), ESHAPE), (dict(n=-1), ESHAPE), (dict(k=-1), ESHAPE), (dict(m=(1 << 31) - 512), ESHAPE),
    (dict(dtype=3), EINVAL), (dict(c=None), EINVAL), (dict(ld_c=199), EINVAL), (dict(c=P + 2), EALIGN),
    # a scale that changes along the contraction
    (dict(ga=COL), EINVAL), (dict(gb=COL), EINVAL), (dict(ta=1, ga=ROW), EINVAL),
    (dict(tb=0, gb=ROW), EINVAL),
    (dict(m=0, c=None), 0), (dict(n=0, c=None), 0), (dict(k=0, acc=1), 0)])
def test_gemm_refusals(lib, change, status):
    change = dict(change)
    a, b = _m(groups=change.pop("ga", ROW)), _m(groups=change.pop("gb", ROW))
    assert _call(lib.mfsdp_gemm_fp8, GEMM, **dict(dict(a=a, b=b), **change)) == status


def test_gemm_takes_both_operands(lib):
    assert _call(lib.mfsdp_gemm_fp8, GEMM, a=None, b=_m()) == EINVAL
    assert _call(lib.mfsdp_gemm_fp8, GEMM, a=_m(), b=None) == EINVAL


NORM_FWD = dict(kind=0, rows=4, cols=64, dtype=1, pdtype=0, x=P, ld_x=64, res=P, ld_r=64, w=P, b=P,
                eps=1e-5, h=P, ld_h=64, y=P, ld_y=64, y8=None, h8=None, mean=P, rstd=P, stream=None)
NORM_BWD = dict(kind=0, rows=4, cols=64, dtype=1, pdtype=0, dy=P, ld_dy=64, dres=P, ld_r=64, h=P, ld_h=64,
                h8=None, w=P, mean=P, rstd=P, dx=P, ld_dx=64, dw=P, db=P, ws=P, ws_bytes=1 << 20,
                stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(kind=2), EINVAL), (dict(dtype=2), EINVAL), (dict(pdtype=-1), EINVAL), (dict(rows=-1), ESHAPE),
    (dict(cols=0), ESHAPE), (dict(cols=1 << 31), ESHAPE), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL), (dict(x=None), EINVAL), (dict(y=None), EINVAL),
    (dict(ld_x=63), EINVAL), (dict(ld_r=63), EINVAL), (dict(ld_h=63), EINVAL), (dict(ld_y=63), EINVAL),
    (dict(kind=1, mean=None), EINVAL), (dict(kind=1, b=None), EINVAL), (dict(x=P + 1), EALIGN),
    (dict(res=P + 1), EALIGN), (dict(h=P + 1), EALIGN), (dict(w=P + 2), EALIGN), (dict(rstd=P + 2), EALIGN),
    (dict(rows=0, x=None), 0)])
def test_norm_forward_refusals(lib, change, status):
    assert _call(lib.mfsdp_norm_residual_forward, NORM_FWD, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(kind=-1), EINVAL), (dict(dtype=5), EINVAL), (dict(rows=1 << 31), ESHAPE), (dict(dy=None), EINVAL),
    (dict(h=None), EINVAL), (dict(dx=None), EINVAL), (dict(rstd=None), EINVAL), (dict(mean=None), EINVAL),
    (dict(ld_dx=10), EINVAL), (dict(ld_r=10), EINVAL), (dict(ld_h=10), EINVAL),
    (dict(kind=1, mean=None), EINVAL), (dict(ws=None), EINVAL), (dict(ws=P + 8), EALIGN),
    (dict(dy=P + 1), EALIGN), (dict(dres=P + 1), EALIGN), (dict(ws_bytes=4 * 2 * 64 * 4 - 1), EWORKSPACE)])
def test_norm_backward_refusals(lib, change, status):
    assert _call(lib.mfsdp_norm_residual_backward, NORM_BWD, **change) == status


def test_norm_backward_takes_one_h(lib):
    assert _call(lib.mfsdp_norm_residual_backward, NORM_BWD, h8=_m()) == EINVAL
    assert _call(lib.mfsdp_norm_residual_backward, NORM_BWD, h=None, h8=_m(groups=COL)) == EINVAL


ACT_FWD = dict(kind=0, rows=4, cols=64, dtype=1, gate=P, ld_g=64, up=P, ld_u=64, y=P, ld_y=64, y8=None,
               gate8=None, up8=None, stream=None)
ACT_BWD = dict(kind=0, rows=4, cols=64, dtype=1, dy=P, ld_dy=64, gate=P, ld_g=64, gate8=None, up=P, ld_u=64,
               up8=None, dgate=P, ld_dg=64, dup=P, ld_du=64, dg_row=None, dg_col=None, du_row=None,
               du_col=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(kind=2), EINVAL), (dict(dtype=2), EINVAL), (dict(rows=-1), ESHAPE), (dict(cols=0), ESHAPE),
    (dict(gate=None), EINVAL), (dict(up=None), EINVAL), (dict(kind=1), EINVAL), (dict(y=None), EINVAL),
    (dict(ld_g=63), EINVAL), (dict(ld_u=63), EINVAL), (dict(ld_y=63), EINVAL), (dict(gate=P + 1), EALIGN),
    (dict(y8="col"), EINVAL), (dict(gate8="tile"), EINVAL), (dict(kind=1, up=None, up8="row"), EINVAL),
    (dict(rows=0, gate=None), 0)])
def test_activation_forward_refusals(lib, change, status):
    kinds = dict(row=ROW, col=COL, tile=TILE)
    change = {k: _m(groups=kinds[v]) if isinstance(v, str) else v for k, v in change.items()}
    assert _call(lib.mfsdp_activation_forward, ACT_FWD, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(kind=3), EINVAL), (dict(dy=None), EINVAL), (dict(gate=None), EINVAL), (dict(up=None), EINVAL),
    (dict(kind=1), EINVAL), (dict(dgate=None, dup=None), EINVAL), (dict(gate8="row"), EINVAL),
    (dict(gate=None, gate8="row"), EINVAL), (dict(dg_row="col"), EINVAL), (dict(dg_col="row"), EINVAL),
    (dict(du_col="tile"), EINVAL), (dict(ld_dg=63), EINVAL), (dict(ld_du=63), EINVAL),
    (dict(ld_dy=63), EINVAL), (dict(dup=P + 1), EALIGN), (dict(rows=0, dy=None), 0)])
def test_activation_backward_refusals(lib, change, status):
    kinds = dict(row=ROW, col=COL, tile=TILE)
    change = {k: _m(groups=kinds[v]) if isinstance(v, str) else v for k, v in change.items()}
    assert _call(lib.mfsdp_activation_backward, ACT_BWD, **change) == status


def test_results_have_buffers_of_their_own(lib):
    """A buffer that two results share, or a result of 8 bits and its source."""
    row, col, tile = _m(), _m(groups=COL), _m(groups=TILE)         # all of the same memory
    assert lib.mfsdp_quantize_fp8(8, 200, 0, P + 4096, 200, row, col, None) == EINVAL
    assert lib.mfsdp_quantize_fp8(8, 200, 0, P, 200, tile, None, None) == EINVAL
    assert lib.mfsdp_regroup_fp8(8, 200, row, tile, None, None) == EINVAL
    assert _call(lib.mfsdp_norm_residual_forward, NORM_FWD) == EINVAL           # h and y
    assert _call(lib.mfsdp_norm_residual_forward, NORM_FWD, h=P + 4096, y8=row) == EINVAL
    assert _call(lib.mfsdp_activation_forward, ACT_FWD, y=None, y8=row, gate8=row) == EINVAL
    assert _call(lib.mfsdp_activation_backward, ACT_BWD) == EINVAL              # dgate and dup
    assert _call(lib.mfsdp_activation_backward, ACT_BWD, dup=None, dgate=P + 4096, dg_row=row,
                 dg_col=col) == EINVAL


# ------------------------------------------------------------------------------------ the binding
def test_binding_refuses_host_tensors_and_shapes():
    from matrix_optimizer_owner_gb300 import mfsdp
    x = torch.zeros(4, 256)
    m = mfsdp.fp8_empty(4, 256, ROW, device="cpu")
    assert m.scales.shape == (4, 2) and m.data.dtype == torch.float8_e4m3fn
    with pytest.raises(ValueError, match="current CUDA device"):
        mfsdp.mfsdp_quantize_fp8(x, m)
    with pytest.raises(ValueError, match="shape"):
        mfsdp.mfsdp_quantize_fp8(torch.zeros(5, 256), m)
    with pytest.raises(TypeError, match="float8"):
        mfsdp.mfsdp_quantize_fp8(x, m._replace(data=x))
    with pytest.raises(TypeError, match="scales"):
        mfsdp.mfsdp_quantize_fp8(x, m._replace(scales=torch.zeros(4, 2)))
    with pytest.raises(ValueError, match="shape"):
        mfsdp.mfsdp_quantize_fp8(x, m._replace(groups=COL))
    with pytest.raises(ValueError, match="groups"):
        mfsdp.mfsdp_quantize_fp8(x, m._replace(groups=7))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        mfsdp.mfsdp_quantize_fp8(x.half(), m)
    with pytest.raises(ValueError, match="expected groups"):
        mfsdp.mfsdp_norm_residual_forward(mfsdp.NORM_RMS, x, None, None, None, 1e-5,
                                          y8=mfsdp.fp8_empty(4, 256, COL, device="cpu"))
    with pytest.raises(ValueError, match="contractions"):
        mfsdp.mfsdp_gemm_fp8(m, mfsdp.fp8_empty(8, 128, ROW, device="cpu"), torch.zeros(4, 8), trans_b=True)


def test_empty_matrix_layout():
    from matrix_optimizer_owner_gb300 import mfsdp
    for rows, cols in ((1, 1), (3, 130), (257, 16), (0, 40)):
        for groups, name in ((ROW, "row"), (COL, "col"), (TILE, "tile")):
            m = mfsdp.fp8_empty(rows, cols, groups, torch.float8_e5m2, device="cpu")
            assert m.data.shape == (rows, cols) and m.data.dtype == torch.float8_e5m2
            assert rows < 2 or m.data.stride(0) % 16 == 0
            assert tuple(m.scales.shape) == oracle.scale_shape(rows, cols, name)


# ------------------------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("kind,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_oracle_rounds_as_float8(kind, dtype):
    gen = torch.Generator().manual_seed(0)
    v = torch.randn(20000, generator=gen) * torch.exp2(torch.randint(-24, 9, (20000,), generator=gen))
    every = torch.arange(256, dtype=torch.uint8).view(dtype).float()
    every = every[every.isfinite()]
    mid = (every[:-1] + every[1:]) / 2                       # ties
    v = torch.cat([v, every, mid[mid.isfinite()]]).clamp(-oracle.TYPES[kind][2], oracle.TYPES[kind][2])
    assert np.array_equal(oracle.round_to(v.numpy(), kind), v.to(dtype).double().numpy())


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_oracle_scales_by_hand(kind):
    big = oracle.TYPES[kind][2]
    x = np.zeros((3, 200))
    x[0, 0], x[0, 150] = big, 2 * big
    x[1, 0] = big * (1 + 1e-9)
    x[2, 5] = np.inf
    q, s = oracle.quantize(x, "row", kind)
    assert s.tolist() == [[127, 128], [128, 0], [0, 0]]
    assert q[0, 0] == big and q[0, 150] == big and q[1, 0] == big / 2 and np.isnan(q[2, 5])
    assert oracle.quantize(x[:2], "tile", kind)[1].tolist() == [[128, 128]]
    assert oracle.quantize(x[:2, :2], "col", kind)[1].tolist() == [[128, 0]]


@pytest.mark.parametrize("kind", ["swiglu", "gelu"])
def test_oracle_gradients(kind):
    """The activations' gradients against torch's functions and automatic differentiation."""
    gen = torch.Generator().manual_seed(1)
    g, u, dy = (torch.randn(500, generator=gen, dtype=torch.float64) * 3 for _ in range(3))
    g.requires_grad_()
    u.requires_grad_()
    y = (torch.nn.functional.silu(g) * u if kind == "swiglu"
         else torch.nn.functional.gelu(g, approximate="tanh") + 0 * u)
    y.backward(dy)
    n = lambda t: t.detach().numpy()  # noqa: E731
    assert np.allclose(oracle.activation(kind, n(g), n(u)), n(y), rtol=1e-12, atol=1e-14)
    dg, du = oracle.activation_grads(kind, n(dy), n(g), n(u))
    assert np.allclose(dg, n(g.grad), rtol=1e-10, atol=1e-13)
    if kind == "swiglu":
        assert np.allclose(du, n(u.grad), rtol=1e-12, atol=1e-14)


def test_struct_matches_the_header():
    """The size of the C structure, by compiling the header."""
    import subprocess
    import tempfile
    from matrix_optimizer_owner_gb300._lib import Fp8Struct
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(src, "w") as f:
            f.write('#include <stdio.h>\n#include <stddef.h>\n#include "mfsdp.h"\nint main(void) { printf("%zu '
                    '%zu %zu", sizeof(mfsdp_fp8_matrix), offsetof(mfsdp_fp8_matrix, scales), '
                    'offsetof(mfsdp_fp8_matrix, groups)); return 0; }\n')
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert got == [str(C.sizeof(Fp8Struct)), str(Fp8Struct.scales.offset), str(Fp8Struct.groups.offset)]
