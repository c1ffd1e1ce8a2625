"""mfsdp_norm_forward / _backward against the float64 oracle.

Tolerances, elementwise, with u = 2^-24: a sum over a row runs at most 32 terms in a thread and
then a tree, so its relative error (against the sum of absolute values) is below 64 u.  With
A = (|x| + mean|x|) r, which bounds |z| and carries the error of the mean,
    |y - y_ref|   <= 64 u (A |w| + |b|)
    |dx - dx_ref| <= 64 u r (|g| + mean|g| + A mean(|g| A))
    |dw - dw_ref| <= (64 + rows) u sum |dy| A         (any order of the sum over the rows)
    |db - db_ref| <= (64 + rows) u sum |dy|
plus the rounding of a result that is stored in bf16 (8 significant bits: 2^-8 of it).  The backward oracle takes the statistics the kernel wrote.
"""

import numpy as np
import pytest
import torch

from oracle import norm as oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _tol(t, ref, base):
    return base + 1e-38 + (np.abs(ref) * 2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0)


def _inputs(rows, cols, dtype, params, layer, seed=0, pitch=0, offset=0, scale=1.0, shift=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def mat(std=1.0, mean=0.0):
        base = torch.randn(rows * (cols + pitch) + offset, generator=gen, device="cuda")
        base = (base * std + mean).to(TYPES[dtype])
        return base[offset:].view(rows, cols + pitch)[:, :cols]

    def vec(mean):
        return (torch.randn(cols, generator=gen, device="cuda") * 0.2 + mean).to(TYPES[params])

    x = mat(scale, shift)
    return x, mat(0.1), vec(1.0), vec(0.0) if layer else None


def _check(rows, cols, dtype="f32", params="f32", layer=True, eps=1e-5, with_w=True, with_b=True,
           **kw):
    from matrix_optimizer_owner_gb300 import mfsdp
    x, dy, w, b = _inputs(rows, cols, dtype, params, layer, **kw)
    w = w if with_w else None
    b = b if with_b and layer else None
    kind = mfsdp.NORM_LAYER if layer else mfsdp.NORM_RMS
    y = torch.full((rows, cols), float("nan"), dtype=x.dtype, device="cuda")
    mean = torch.full((rows,), float("nan"), device="cuda") if layer else None
    rstd = torch.full((rows,), float("nan"), device="cuda")
    mfsdp.mfsdp_norm_forward(kind, x, w, b, eps, y, mean, rstd)
    X, DY, W, B = _np(x), _np(dy), _np(w), _np(b)
    ref, mu, r = oracle.forward(X, W, B, eps, layer)
    aw = np.abs(W) if w is not None else np.ones(cols)
    A = (np.abs(X) + np.abs(X).mean(1, keepdims=True)) * r[:, None]
    base = 64 * U * (A * aw + (np.abs(B) if b is not None else 0.0))
    assert (np.abs(_np(y) - ref) <= _tol(y, ref, base)).all()
    if layer:
        assert (np.abs(_np(mean) - mu) <= 64 * U * np.abs(X).mean(1) + 1e-38).all()
    # d log r = r^2 d var / 2, and var carries the mean's error through x
    assert (np.abs(_np(rstd) - r) <= 64 * U * r * (1 + (A * A).mean(1))).all()

    dx = torch.full((rows, cols), float("nan"), dtype=x.dtype, device="cuda")
    vec = (lambda: torch.full((cols,), float("nan"), dtype=TYPES[params], device="cuda"))
    dw, db = vec(), vec() if layer else None
    mfsdp.mfsdp_norm_backward(kind, dy, x, w, mean, rstd, dx, dw, db)
    M, R = (_np(mean) if layer else np.zeros(rows)), _np(rstd)
    rdx, rdw, rdb = oracle.backward(DY, X, W, M, R, layer)
    A = (np.abs(X) + np.abs(M)[:, None]) * R[:, None]
    G = np.abs(DY) * aw
    base = 64 * U * R[:, None] * (G + G.mean(1, keepdims=True) + A * (G * A).mean(1, keepdims=True))
    assert (np.abs(_np(dx) - rdx) <= _tol(dx, rdx, base)).all()
    base = (64 + rows) * U * (np.abs(DY) * A).sum(0)
    assert (np.abs(_np(dw) - rdw) <= _tol(dw, rdw, base)).all()
    if layer:
        base = (64 + rows) * U * np.abs(DY).sum(0)
        assert (np.abs(_np(db) - rdb) <= _tol(db, rdb, base)).all()
    return x, dy, w, b, mean, rstd, dx, dw, db


# one warp per row with 1-4 chunks, block rows of every size, rows of passes; one column
@pytest.mark.parametrize("cols", [1, 7, 8, 33, 256, 257, 512, 768, 1000, 1024, 1025, 2048, 4096,
                                  5120, 8192, 8193, 16384, 20000, 32768, 40000])
@pytest.mark.parametrize("dtype,layer", [("f32", True), ("bf16", False)])
def test_widths(cols, dtype, layer):
    _check(5, cols, dtype, "f32", layer)


@pytest.mark.parametrize("rows", [1, 8, 9, 300])
@pytest.mark.parametrize("cols", [192, 1100])
@pytest.mark.parametrize("dtype,params", [("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_rows_and_types(rows, cols, dtype, params):
    _check(rows, cols, dtype, params, True, seed=1)


def test_more_rows_than_blocks():
    _check(20011, 64, "f32", "f32", True, seed=2)
    _check(6007, 1536, "bf16", "f32", False, seed=3)


@pytest.mark.parametrize("pitch,offset", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_offsets(pitch, offset, dtype):
    _check(37, 264, dtype, "f32", True, seed=4, pitch=pitch, offset=offset)


@pytest.mark.parametrize("with_w,with_b", [(False, True), (True, False), (False, False)])
def test_absent_parameters(with_w, with_b):
    _check(11, 320, "f32", "f32", True, seed=5, with_w=with_w, with_b=with_b)


def test_large_mean_does_not_cancel():
    # the mean is 1000 standard deviations off: summing squares would lose every digit
    _check(9, 768, "f32", "f32", True, seed=6, scale=0.01, shift=10.0)


def test_constant_rows_and_eps():
    from matrix_optimizer_owner_gb300 import mfsdp
    x = torch.full((3, 100), 2.5, device="cuda")
    b = torch.arange(100, device="cuda", dtype=torch.float32)
    y, rstd, mean = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x, None, b, 1e-4, y, mean, rstd)
    assert torch.equal(y, b.expand(3, 100)) and torch.allclose(rstd, torch.full_like(rstd, 100.0))


def test_rows_with_nan_stay_apart():
    from matrix_optimizer_owner_gb300 import mfsdp
    x, dy, w, b = _inputs(6, 128, "f32", "f32", True, seed=7)
    clean = torch.empty_like(x)
    mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x, w, b, 1e-5, clean)
    bad = x.clone()
    bad[2, 5], bad[4, 0] = float("nan"), float("inf")
    y = torch.empty_like(x)
    mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, bad, w, b, 1e-5, y)
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], clean[keep]) and y[[2, 4]].isnan().all()


def test_in_place_and_repeatable():
    from matrix_optimizer_owner_gb300 import mfsdp
    x, dy, w, b, mean, rstd, dx, dw, db = _check(700, 768, "bf16", "f32", True, seed=8)
    again, dw2, db2 = dy.clone(), torch.empty_like(dw), torch.empty_like(db)
    mfsdp.mfsdp_norm_backward(mfsdp.NORM_LAYER, again, x, w, mean, rstd, again, dw2, db2)
    assert torch.equal(again, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    y, inplace = torch.empty_like(x), x.clone()
    mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x, w, b, 1e-5, y)
    mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, inplace, w, b, 1e-5, inplace)
    assert torch.equal(y, inplace)


def test_no_rows():
    from matrix_optimizer_owner_gb300 import mfsdp
    x = torch.empty(0, 40, device="cuda")
    dw, db = torch.full((40,), 3.0, device="cuda"), torch.full((40,), 3.0, device="cuda")
    stats = torch.empty(0, device="cuda")
    mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x, None, None, 1e-5, x, stats, stats)
    mfsdp.mfsdp_norm_backward(mfsdp.NORM_LAYER, x, x, None, stats, stats, x, dw, db)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("layer", [True, False])
def test_gradient_against_differences(layer):
    """<dx, v> and <dw, v> against central differences of L = <y, dy>, extrapolated from steps h
    and h / 2.  The extrapolation's error is below the difference of the two quotients; the
    rounding of y adds 64 u sum(A |w| + |b|) |dy| / (h / 2) per quotient, twice in all."""
    from matrix_optimizer_owner_gb300 import mfsdp
    x, dy, w, b, mean, rstd, dx, dw, db = _check(4, 96, "f32", "f32", layer, seed=9)
    kind = mfsdp.NORM_LAYER if layer else mfsdp.NORM_RMS
    gen = torch.Generator(device="cuda").manual_seed(10)

    def loss(xx, ww):
        y = torch.empty_like(x)
        mfsdp.mfsdp_norm_forward(kind, xx, ww, b, 1e-5, y)
        return float((y.double() * dy.double()).sum())

    X, W, B = _np(x), np.abs(_np(w)), (np.abs(_np(b)) if layer else 0.0)
    A = (np.abs(X) + np.abs(X).mean(1, keepdims=True)) * _np(rstd)[:, None]
    noise = 64 * U * ((A * W + B) * np.abs(_np(dy))).sum()
    for which, grad in (("x", dx), ("w", dw)):
        v = torch.randn(grad.shape, generator=gen, device="cuda")
        quot = []
        for h in (2.0 ** -6, 2.0 ** -7):
            if which == "x":
                quot.append((loss(x + h * v, w) - loss(x - h * v, w)) / (2 * h))
            else:
                quot.append((loss(x, w + h * v) - loss(x, w - h * v)) / (2 * h))
        want = (4 * quot[1] - quot[0]) / 3
        got = float((grad.double() * v.double()).sum())
        # x + h v is rounded to fp32: an error u (|x| + h) in x moves L by u sum |dx| (|x| + h)
        moved = 4 * U * float((dx.double().abs() * (x.double().abs() + 1)).sum()) * 2 ** 7
        assert abs(got - want) <= abs(quot[1] - quot[0]) + 4 * noise * 2 ** 7 + moved


def test_other_stream_and_graph():
    from matrix_optimizer_owner_gb300 import mfsdp
    x, dy, w, b, mean, rstd, dx, dw, db = _check(64, 512, "bf16", "f32", True, seed=11)
    ws = torch.empty(mfsdp.mfsdp_norm_backward_workspace_bytes(64, 512), dtype=torch.uint8,
                     device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    mfsdp.mfsdp_norm_backward(mfsdp.NORM_LAYER, dy, x, w, mean, rstd, dx2, dw2, db2, stream=s)
    s.synchronize()
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    dx2.zero_(), dw2.zero_(), db2.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mfsdp.mfsdp_norm_backward(mfsdp.NORM_LAYER, dy, x, w, mean, rstd, dx2, dw2, db2, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
