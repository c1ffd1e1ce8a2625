"""The 8-bit operators together, as ``examples/train_fp8_feed_forward.py`` runs them, and in CUDA graphs, on
other streams, from several threads and on buffers of more than 2^31 elements.

Against the same block in float64 with the same roundings.  A value that lies within the fp32 error of a
border may be rounded the other way, a step (2^-2 of it in e5m2) off; where a thousandth of an operand's
values are, a product's relative error (Frobenius) is at most sqrt(1e-3) 2^-2 = 8e-3, and with up to three
such operands on a gradient's way 1.4e-2; a bf16 result adds 2^-9.
"""

import threading

import numpy as np
import pytest
import torch

from oracle import fp8 as oracle
from oracle import norm as onorm

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().double().cpu().numpy()


def _bf(a):
    return torch.tensor(np.asarray(a)).to(torch.bfloat16).double().numpy()


def _q(v, groups, kind="e4m3"):
    q, s = oracle.quantize(v, groups, kind)
    return oracle.values(q, s, groups)


def _rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def _model(dim=256, hidden=640, tokens=300):
    import examples.train_fp8_feed_forward as ex
    m = ex.FeedForward(dim, hidden, tokens)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(tokens, dim, generator=gen, device="cuda").bfloat16() for _ in range(2))
    dout = (torch.randn(tokens, dim, generator=gen, device="cuda") * 1e-3).bfloat16()
    m.norm_w.copy_(1 + 0.1 * torch.randn(dim, generator=gen, device="cuda"))
    return m, x, r, dout


def test_block_against_float64():
    m, x, r, dout = _model()
    out = _np(m.forward(x, r))
    dx = _np(m.backward(dout))
    X, R, D, w = _np(x), _np(r), _np(dout), _np(m.norm_w)
    W = {k: _q(_np(v), "tile") for k, v in m.w.items()}
    H = X + R
    Y, _, rstd = onorm.forward(H, w, None, m.eps, False)
    y = _q(Y, "row")
    gate, up = _bf(y @ W["gate"].T), _bf(y @ W["up"].T)
    z = _q(oracle.activation("swiglu", gate, up), "row")
    assert _rel(out, _bf(H) + z @ W["down"].T) <= 1.4e-2 + 2.0 ** -9
    gk, uk, hk = _q(gate, "row"), _q(up, "row"), _q(H, "row")
    g_down = _q(D, "col", "e5m2").T @ _q(z, "col")
    dz = _bf(_q(D, "row", "e5m2") @ W["down"])
    dg, du = oracle.activation_grads("swiglu", dz, gk, uk)
    yc = _q(y, "col")
    g_gate = _q(dg, "col", "e5m2").T @ yc
    g_up = _q(du, "col", "e5m2").T @ yc
    dy = _bf(_bf(_q(dg, "row", "e5m2") @ W["gate"]) + _q(du, "row", "e5m2") @ W["up"])
    DX, DW, _ = onorm.backward(dy, hk, w, np.zeros(len(H)), rstd, False)
    for got, want in ((_np(m.g["down"]), g_down), (_np(m.g["gate"]), g_gate), (_np(m.g["up"]), g_up),
                      (dx, DX + D), (_np(m.norm_grad), DW)):
        assert _rel(got, want) <= 1.4e-2 + 2.0 ** -9


def test_block_gradients_against_differences():
    """Against the block without any rounding: directional derivatives of sum(out dout) in float64.  A
    rounding to 8 bits is at most 2^-4 (e4m3) or 2^-3 (e5m2) of a value, uniform: 2^-4 / sqrt(3) = 0.036 and
    0.072 rms.  A gradient here passes up to six e4m3 roundings (y, W, gate, up, z, h) and two e5m2 ones, of
    independent values: sqrt(6 0.036^2 + 2 0.072^2) = 0.135 of the gradient's norm, and a direction that is
    the gradient itself shows only the part of that error along it."""
    m, x, r, dout = _model()
    m.forward(x, r)
    dx = _np(m.backward(dout))
    X, R, D, w = _np(x), _np(r), _np(dout), _np(m.norm_w)
    W = {k: _np(v).copy() for k, v in m.w.items()}

    def value(W, w, X):
        H = X + R
        Y, _, _ = onorm.forward(H, w, None, m.eps, False)
        Z = oracle.activation("swiglu", Y @ W["gate"].T, Y @ W["up"].T)
        return float(((H + Z @ W["down"].T) * D).sum())

    for name in W:
        g = _np(m.g[name])
        t = 1e-4 * np.linalg.norm(W[name]) / np.linalg.norm(g)
        up, down = (value(dict(W, **{name: W[name] + s * t * g}), w, X) for s in (1, -1))
        assert abs((up - down) / (2 * t) / (g * g).sum() - 1) <= 0.135
    g = _np(m.norm_grad)
    t = 1e-4 * np.linalg.norm(w) / np.linalg.norm(g)
    assert abs((value(W, w + t * g, X) - value(W, w - t * g, X)) / (2 * t) / (g * g).sum() - 1) <= 0.135
    t = 1e-4 * np.linalg.norm(X) / np.linalg.norm(dx)
    assert abs((value(W, w, X + t * dx) - value(W, w, X - t * dx)) / (2 * t) / (dx * dx).sum() - 1) <= 0.135


def test_gradients_reach_the_owner_step():
    """The matrices' gradients are the owner step's contribution: its reduced gradient, bit for bit."""
    from matrix_optimizer_owner_gb300 import mfsdp
    from workloads.configs import Hyper
    m, x, r, dout = _model()
    before = m.owner.weights.clone()
    m.forward(x, r)
    m.backward(dout)
    reduced = torch.zeros_like(m.grad)
    m.owner.step([m.grad], [m.norm_grad], Hyper(), reduced_grad=reduced)
    assert torch.equal(reduced, m.grad) and not torch.equal(before, m.owner.weights)
    assert mfsdp.mfsdp_query_status() == 0 and m.owner.weights.isfinite().all()


def test_example_runs():
    import sys
    from unittest import mock

    import examples.train_fp8_feed_forward as ex
    with mock.patch.object(sys, "argv", ["x", "--steps", "3", "--tokens", "200"]):
        ex.main()


def test_block_captured_and_replayed():
    """Forward and backward in one graph, replayed on new inputs, beside eager runs of the same buffers'
    twins."""
    a, x, r, dout = _model()
    b = _model()[0]
    b.forward(x, r)
    b.backward(dout)                                   # loads the kernels
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.forward(x, r)
        b.backward(dout)
    gen = torch.Generator(device="cuda").manual_seed(9)
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        dout.copy_(torch.randn(x.shape, generator=gen, device="cuda") * 1e-3)
        b.grad.zero_()
        g.replay()
        a.forward(x, r)
        a.backward(dout)
        torch.cuda.synchronize()
        for n in ("out", "dx", "grad", "norm_grad"):
            assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_block_on_streams_and_threads():
    """Blocks of their own, run at the same time from several host threads."""
    models = [_model() for _ in range(3)]
    want = []
    for m, x, r, dout in models:
        m.forward(x, r)
        want.append((m.backward(dout).clone(), m.grad.clone()))
    torch.cuda.synchronize()
    got = [None] * 3

    def work(i):
        torch.cuda.set_device(0)
        m, x, r, dout = models[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                m.forward(x, r)
                m.backward(dout)
            got[i] = (m.dx.clone(), m.grad.clone())
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for (a, b), (c, d) in zip(got, want):
        assert torch.equal(a, c) and torch.equal(b, d)


def test_explicit_stream():
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(300, 520, generator=gen, device="cuda")
    s = torch.cuda.Stream()
    a, b = mfsdp.fp8_empty(300, 520, 0), mfsdp.fp8_empty(300, 520, 1)
    w = mfsdp.fp8_empty(300, 520, 2)
    y, y2 = torch.empty(300, 300, device="cuda"), torch.empty(300, 300, device="cuda")
    back = torch.empty_like(x)
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        mfsdp.mfsdp_quantize_fp8(x, a, b, stream=stream)
        mfsdp.mfsdp_regroup_fp8(a, w, stream=stream)
        mfsdp.mfsdp_gemm_fp8(a, w, y, trans_b=True, stream=stream)
        mfsdp.mfsdp_dequantize_fp8(a, back, stream=stream)
    s.synchronize()
    mfsdp.mfsdp_gemm_fp8(a, w, y2, trans_b=True)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and (back - x).abs().max() <= x.abs().max() / 16


# ------------------------------------------------------------------------------------ far offsets
def _same8(a, b):
    u = lambda t: t.view(torch.uint8)  # noqa: E731
    return torch.equal(u(a.data), u(b.data)) and torch.equal(u(a.scales), u(b.scales))


def _tail(m, rows):
    from matrix_optimizer_owner_gb300 import mfsdp
    n = rows if m.groups == 0 else -(-rows // 128)
    return mfsdp.Fp8Matrix(m.data[-rows:], m.scales[-n:], m.groups)


def test_rows_past_32_bit_offsets():
    """The last rows of matrices of more than 2^31 elements come out as they do alone."""
    from matrix_optimizer_owner_gb300 import mfsdp
    rows, cols, tail = 262144 + 1280, 8192, 256       # 2.16e9 elements
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-tail:] = torch.randn(tail, cols, generator=gen, device="cuda")
    small = x[-tail:].clone()
    new = lambda n, g: mfsdp.fp8_empty(n, cols, g)  # noqa: E731
    big8, big8c, one, onec = new(rows, 0), new(rows, 1), new(tail, 0), new(tail, 1)
    mfsdp.mfsdp_quantize_fp8(x, big8, big8c)
    mfsdp.mfsdp_quantize_fp8(small, one, onec)
    assert _same8(_tail(big8, tail), one) and _same8(_tail(big8c, tail), onec)
    big8c.data.view(torch.uint8).zero_()
    mfsdp.mfsdp_regroup_fp8(big8, big8c)
    mfsdp.mfsdp_regroup_fp8(one, onec)
    assert _same8(_tail(big8c, tail), onec)
    del big8c
    w = mfsdp.fp8_empty(256, cols, 2)
    mfsdp.mfsdp_quantize_fp8(torch.randn(256, cols, generator=gen, device="cuda"), w)
    y, y1 = (torch.empty(n, 256, dtype=torch.bfloat16, device="cuda") for n in (rows, tail))
    mfsdp.mfsdp_gemm_fp8(big8, w, y, trans_b=True)
    mfsdp.mfsdp_gemm_fp8(one, w, y1, trans_b=True)
    # (other tiles, so other orders of the same sums: half a bf16 step and the sums' own errors)
    assert (y[-tail:].float() - y1.float()).abs().max() <= 2.0 ** -7 * y1.float().abs().max()
    assert not y[:-tail].any()
    del y
    rstd, rstd1 = torch.empty(rows, device="cuda"), torch.empty(tail, device="cuda")
    h = torch.empty_like(x)
    mfsdp.mfsdp_norm_residual_forward(mfsdp.NORM_RMS, x, x, None, None, 1e-6, h=h, y8=big8, rstd=rstd)
    h1 = torch.empty_like(small)
    mfsdp.mfsdp_norm_residual_forward(mfsdp.NORM_RMS, small, small, None, None, 1e-6, h=h1, y8=one,
                                      rstd=rstd1)
    assert torch.equal(h[-tail:], h1) and _same8(_tail(big8, tail), one)
    dx1 = torch.empty_like(small)
    mfsdp.mfsdp_norm_residual_backward(mfsdp.NORM_RMS, x, x, h, None, None, rstd, h)
    mfsdp.mfsdp_norm_residual_backward(mfsdp.NORM_RMS, small, small, h1, None, None, rstd1, dx1)
    assert torch.equal(h[-tail:], dx1)
    mfsdp.mfsdp_activation_forward(mfsdp.ACT_GELU, x, None, y=h, y8=big8)
    mfsdp.mfsdp_activation_forward(mfsdp.ACT_GELU, small, None, y=h1, y8=one)
    assert torch.equal(h[-tail:], h1) and _same8(_tail(big8, tail), one)
    mfsdp.mfsdp_activation_backward(mfsdp.ACT_GELU, x, x, None, dgate=h, dgate8=big8)
    mfsdp.mfsdp_activation_backward(mfsdp.ACT_GELU, small, small, None, dgate=h1, dgate8=one)
    assert torch.equal(h[-tail:], h1) and _same8(_tail(big8, tail), one)


def test_gemm_output_past_32_bit_offsets():
    from matrix_optimizer_owner_gb300 import mfsdp
    m, n, k = 40000, 60000, 128                        # 2.4e9 entries
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, b = mfsdp.fp8_empty(m, k, 0), mfsdp.fp8_empty(n, k, 0)
    mfsdp.mfsdp_quantize_fp8(torch.randn(m, k, generator=gen, device="cuda"), a)
    mfsdp.mfsdp_quantize_fp8(torch.randn(n, k, generator=gen, device="cuda"), b)
    c = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    mfsdp.mfsdp_gemm_fp8(a, b, c, trans_b=True)
    va, vb = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
    mfsdp.mfsdp_dequantize_fp8(a, va)
    mfsdp.mfsdp_dequantize_fp8(b, vb)
    for rows in (slice(0, 100), slice(m - 300, m)):
        ref = va[rows].double() @ vb.double().T
        tol = (k / 32 + 8) * 2.0 ** -22 * (va[rows].double().abs() @ vb.double().abs().T)
        assert ((c[rows].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2 * tol).all()
    assert mfsdp.mfsdp_query_status() == 0
