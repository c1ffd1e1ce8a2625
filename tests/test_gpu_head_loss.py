"""mfsdp_head_loss_forward / _backward against the float64 oracle.

Tolerances, elementwise.  A logit is a sum of K products, S = sum |h w|:
  bf16  the products are exact; the tensor cores add them 16 at a time into fp32 without
        rounding to nearest: |dz| <= (K / 16 + 8) 2^-22 S
  fp32  3xTF32: 2^-20 per product and 12 accumulations per block of 32, blocks added in fp32:
        |dz| <= (2^-18 + K / 32 2^-24) S
so lse, a weighted mean of the logits' errors, is off by at most max_v |dz| plus the sum's own
rounding, 2^-18 (1 + |lse|); loss adds |dz| of the label and one rounding.  An entry of G has
relative error 2 max|dz| + 2^-19 (1 + |z| + |lse|) in its probability and, in bf16, is rounded
(bf16 holds 8 significant bits: to nearest is within 2^-8 of the value).  The gradients add up
those errors against the other factor, their own accumulation as above with K = vocab or tokens,
and a bf16 result's rounding (2^-8 of it).
"""

import numpy as np
import pytest
import torch

from oracle import head_loss as oracle

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


def _acc(k, dtype):
    return (k / 16 + 8) * 2.0 ** -22 if dtype == "bf16" else 2.0 ** -18 + k / 32 * 2.0 ** -24


def _mat(rows, cols, dtype, gen, std=1.0, pitch=0, offset=0):
    base = torch.randn(rows * (cols + pitch) + offset, generator=gen, device="cuda") * std
    return base.to(TYPES[dtype])[offset:].view(rows, cols + pitch)[:, :cols]


def _case(n, dim, vocab, dtype="bf16", ignored=0.2, index=torch.int64, seed=0, pitch=0, offset=0,
          std=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = _mat(n, dim, dtype, gen, 1.0, pitch, offset)
    w = _mat(vocab, dim, dtype, gen, std or 2.0 / dim ** 0.5, pitch, offset)
    lab = torch.randint(vocab, (n,), generator=gen, device="cuda")
    lab[torch.rand(n, generator=gen, device="cuda") < ignored] = -100
    dl = torch.rand(n, generator=gen, device="cuda") / max(n, 1) - 0.3 / max(n, 1)
    return h, w, lab.to(index), dl


def _run(h, w, lab, dl, ignore=-100, piece=0, want=("h", "w"), dh=None, dw=None):
    from matrix_optimizer_owner_gb300 import mfsdp
    n = h.shape[0]
    loss, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    mfsdp.mfsdp_head_loss_forward(h, w, lab, loss, lse, ignore_index=ignore)
    if dh is None:
        dh = torch.full(h.shape, float("nan"), dtype=h.dtype, device="cuda")
    if dw is None:
        dw = torch.full(w.shape, float("nan"), dtype=w.dtype, device="cuda")
    mfsdp.mfsdp_head_loss_backward(h, w, lab, lse, dl, dh if "h" in want else None,
                                   dw if "w" in want else None, ignore_index=ignore, piece=piece)
    return loss, lse, dh, dw


def _verify(h, w, lab, dl, out, ignore=-100):
    loss, lse, dh, dw = out
    dtype = "bf16" if h.dtype == torch.bfloat16 else "f32"
    n, dim = h.shape
    vocab = w.shape[0]
    H, W, L, D = _np(h), _np(w), lab.cpu().numpy(), _np(dl)
    rows = oracle.live_rows(L, vocab, ignore)
    H[np.setdiff1d(np.arange(n), rows)] = 0.0     # what dropped rows hold does not matter
    rloss, rlse = oracle.forward(H, W, L, ignore)
    at = (np.arange(len(rows)), L[rows])
    dz = _acc(dim, dtype) * (np.abs(H[rows]) @ np.abs(W).T)
    dlse = dz.max(axis=1) + 2.0 ** -18 * (1 + np.abs(rlse[rows])) if len(rows) else np.zeros(0)
    z = H[rows] @ W.T
    dloss_tol = dlse + dz[at] + 2.0 ** -23 * (np.abs(rlse[rows]) + np.abs(z[at]))
    full = np.zeros(n)
    full[rows] = dlse
    assert (np.abs(_np(lse) - rlse) <= full).all()
    full[rows] = dloss_tol
    assert (np.abs(_np(loss) - rloss) <= full).all()
    _, G = oracle.logit_gradient(H, W, L, D, ignore)
    p = np.exp(z - rlse[rows][:, None])
    rel = 2 * (dz.max(axis=1) + dlse)[:, None] if len(rows) else 0.0
    dG = p * np.abs(D[rows])[:, None] * (rel + 2.0 ** -19 * (1 + np.abs(z) + np.abs(rlse[rows])[:, None]))
    dG = dG + np.abs(G) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22)
    rdh, rdw = oracle.backward(H, W, L, D, ignore)
    aG = np.abs(G) + dG
    out_round = 2.0 ** -8 if dtype == "bf16" else 0.0
    tol = np.zeros(H.shape)
    tol[rows] = dG @ np.abs(W) + _acc(vocab, dtype) * (aG @ np.abs(W))
    assert (np.abs(_np(dh) - rdh) <= tol + out_round * np.abs(rdh) + 1e-38).all()
    tol = dG.T @ np.abs(H[rows]) + _acc(n, dtype) * (aG.T @ np.abs(H[rows]))
    assert (np.abs(_np(dw) - rdw) <= tol + out_round * np.abs(rdw) + 1e-38).all()


# tile and k-block boundaries, one token, one column, odd sizes
@pytest.mark.parametrize("n,dim,vocab", [
    (1, 64, 1000), (2, 1, 300), (7, 768, 513), (64, 64, 64), (255, 72, 255), (256, 128, 256),
    (257, 200, 257), (300, 100, 1031), (513, 320, 2049), (3, 1030, 1), (40, 136, 4000),
    (700, 320, 9001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes(n, dim, vocab, dtype):
    h, w, lab, dl = _case(n, dim, vocab, dtype, ignored=0.2 if n > 2 else 0.0, seed=n)
    _verify(h, w, lab, dl, _run(h, w, lab, dl))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("piece", [1, 256, 768, 5000])
def test_pieces(dtype, piece):
    h, w, lab, dl = _case(300, 96, 2100, dtype, seed=piece)
    _verify(h, w, lab, dl, _run(h, w, lab, dl, piece=piece))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pitch,offset", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 3)])
def test_strides_and_offsets(dtype, pitch, offset):
    h, w, lab, dl = _case(130, 104, 900, dtype, seed=pitch + offset, pitch=pitch, offset=offset)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dh = _mat(130, 104, dtype, gen, 1.0, pitch, offset)
    dw = _mat(900, 104, dtype, gen, 1.0, pitch, offset)
    out = _run(h, w, lab, dl, dh=dh, dw=dw)
    _verify(h, w, lab, dl, out)
    # unaligned weights are copied in pieces
    _verify(h, w, lab, dl, _run(h, w, lab, dl, piece=256))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ignored_tokens(dtype):
    from matrix_optimizer_owner_gb300 import mfsdp
    for ignored, index, ignore in ((0.0, torch.int32, -100), (0.97, torch.int64, -100),
                                   (1.0, torch.int32, -100)):
        h, w, lab, dl = _case(400, 64, 600, dtype, ignored, index, seed=3)
        out = _run(h, w, lab, dl, ignore=ignore)
        _verify(h, w, lab, dl, out, ignore)
        if ignored == 1.0:
            assert not any(t.any().item() for t in out)
    # an ignore index inside the vocabulary, and none in use
    h, w, lab, dl = _case(200, 64, 20, dtype, 0.0, seed=4)
    _verify(h, w, lab, dl, _run(h, w, lab, dl, ignore=7), 7)
    assert mfsdp.mfsdp_query_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropped_rows_may_hold_anything(dtype):
    from matrix_optimizer_owner_gb300 import _lib, mfsdp
    h, w, lab, dl = _case(300, 80, 700, dtype, 0.3, seed=5)
    drop = lab == -100
    h[drop] = float("nan")
    dl[drop] = float("inf")
    out = _run(h, w, lab, dl)
    dl[drop] = 0.0
    _verify(h, w, lab, dl, out)
    assert mfsdp.mfsdp_query_status() == 0
    lab[:4] = torch.tensor([700, -1, 1 << 20, 699], device="cuda")
    h[:4] = 1.0
    out = _run(h, w, lab, dl)
    assert _lib.STATUS_NAMES[mfsdp.mfsdp_query_status()] == "MFSDP_EINDEX"
    _verify(h, w, lab, dl, out)
    assert not out[0][:3].any() and out[0][3] != 0


# fp32 products on either side of what the CUDA cores take (2^29 operations): tiles of 32 and steps
# of 64 that end inside, one token, many tokens, slices of dH, and the same beyond, on 3xTF32
@pytest.mark.parametrize("n,dim,vocab", [
    (5, 65, 33), (31, 64, 32), (33, 63, 65), (1, 300, 5000), (129, 1, 129), (2000, 33, 700),
    (60, 1000, 2050), (520, 520, 1100), (40, 1400, 5000), (2100, 130, 1300)])
@pytest.mark.parametrize("piece", [0, 300])
def test_f32_small_and_large(n, dim, vocab, piece):
    h, w, lab, dl = _case(n, dim, vocab, "f32", 0.2 if n > 1 else 0.0, seed=n + dim)
    _verify(h, w, lab, dl, _run(h, w, lab, dl, piece=piece))


@pytest.mark.parametrize("n,dim,vocab", [(100, 72, 500), (540, 520, 1000)])
@pytest.mark.parametrize("pitch,offset", [(8, 8), (3, 0), (0, 1)])
def test_f32_strides_small_and_large(n, dim, vocab, pitch, offset):
    h, w, lab, dl = _case(n, dim, vocab, "f32", seed=pitch + offset, pitch=pitch, offset=offset)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dh = _mat(n, dim, "f32", gen, 1.0, pitch, offset)
    dw = _mat(vocab, dim, "f32", gen, 1.0, pitch, offset)
    _verify(h, w, lab, dl, _run(h, w, lab, dl, piece=512, dh=dh, dw=dw))


@pytest.mark.parametrize("n,dim,vocab", [(100, 72, 500), (540, 520, 1000)])
def test_f32_dropped_small_and_large(n, dim, vocab):
    from matrix_optimizer_owner_gb300 import mfsdp
    h, w, lab, dl = _case(n, dim, vocab, "f32", 0.4, torch.int32, seed=12)
    drop = lab == -100
    h[drop] = float("nan")
    dl[drop] = float("nan")
    out = _run(h, w, lab, dl, piece=256)
    dl[drop] = 0.0
    _verify(h, w, lab, dl, out)
    again = _run(h, w, lab, dl, piece=256)
    assert all(torch.equal(a, b) for a, b in zip(again, out))
    lab[:] = -100
    assert not any(t.any().item() for t in _run(h, w, lab, dl, piece=256))
    assert mfsdp.mfsdp_query_status() == 0


# the backward pass of up to four tokens: one pass over W, more rows than its blocks take at once,
# odd widths, and widths whose sums do not fit beside it
@pytest.mark.parametrize("n", [1, 2, 3, 4])
@pytest.mark.parametrize("dim,vocab", [(1, 1), (3, 17), (64, 16), (130, 5000), (1024, 9999),
                                       (6400, 300), (6408, 300), (13000, 200)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_tokens_backward(n, dim, vocab, dtype):
    h, w, lab, dl = _case(n, dim, vocab, dtype, 0.0, torch.int32, seed=n + dim)
    if n > 2:
        lab[1] = -100
        h[1] = float("nan")
        dl[1] = float("nan")
    out = _run(h, w, lab, dl)
    if n > 2:
        dl[1] = 0.0
    _verify(h, w, lab, dl, out)
    again = _run(h, w, lab, dl)
    assert all(torch.equal(a, b) for a, b in zip(again, out))
    assert torch.equal(_run(h, w, lab, dl, want="h")[2], out[2])
    assert torch.equal(_run(h, w, lab, dl, want="w")[3], out[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pitch,offset", [(8, 0), (4, 4), (3, 0), (0, 1)])
def test_few_tokens_backward_strides(dtype, pitch, offset):
    h, w, lab, dl = _case(3, 104, 3000, dtype, 0.0, seed=pitch + offset, pitch=pitch, offset=offset)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dh = _mat(3, 104, dtype, gen, 1.0, pitch, offset)
    dw = _mat(3000, 104, dtype, gen, 1.0, pitch, offset)
    _verify(h, w, lab, dl, _run(h, w, lab, dl, dh=dh, dw=dw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_tokens_backward_bad_label_and_infinite_weight(dtype):
    from matrix_optimizer_owner_gb300 import _lib, mfsdp
    h, w, lab, dl = _case(3, 100, 700, dtype, 0.0, seed=16)
    lab[1] = 700
    w[5, 7] = float("inf")
    _, _, dh, _ = _run(h, w, lab, dl)
    assert not dh[1].any()                           # a dropped token, whatever W holds
    assert _lib.STATUS_NAMES[mfsdp.mfsdp_query_status()] == "MFSDP_EINDEX"
    inplace = h.clone()
    w[5, 7] = 0.0
    loss, lse, dh, dw = _run(h, w, lab, dl)
    mfsdp.mfsdp_head_loss_backward(inplace, w, lab, lse, dl, inplace, dw)
    assert torch.equal(inplace, dh)
    mfsdp.mfsdp_query_status()


# bf16 products that the tensor cores take (above 64 Mi operations): tiles, k-blocks and pieces
# that end inside, few tokens, rows that TMA cannot read
@pytest.mark.parametrize("n,dim,vocab", [
    (255, 520, 515), (256, 512, 512), (257, 584, 513), (513, 72, 2049), (5, 1030, 2000),
    (64, 64, 13000), (33, 1100, 1025), (1025, 320, 255), (2, 2049, 2000), (1, 3300, 1000),
    (3, 1088, 2000), (4, 2048, 777)])
@pytest.mark.parametrize("piece", [0, 256])
def test_bf16_tensor_core_sizes(n, dim, vocab, piece):
    h, w, lab, dl = _case(n, dim, vocab, "bf16", 0.2 if n > 2 else 0.0, seed=n + dim)
    _verify(h, w, lab, dl, _run(h, w, lab, dl, piece=piece))


@pytest.mark.parametrize("pitch,offset", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 3)])
def test_bf16_tensor_core_strides(pitch, offset):
    h, w, lab, dl = _case(270, 328, 900, "bf16", seed=pitch + offset, pitch=pitch, offset=offset)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dh = _mat(270, 328, "bf16", gen, 1.0, pitch, offset)
    dw = _mat(900, 328, "bf16", gen, 1.0, pitch, offset)
    for piece in (0, 256):
        _verify(h, w, lab, dl, _run(h, w, lab, dl, piece=piece, dh=dh, dw=dw))


def test_bf16_tensor_core_dropped_rows():
    from matrix_optimizer_owner_gb300 import mfsdp
    for ignored in (0.3, 0.97, 1.0):
        h, w, lab, dl = _case(400, 264, 1100, "bf16", ignored, torch.int32, seed=14)
        drop = lab == -100
        h[drop] = float("nan")
        dl[drop] = float("inf")
        out = _run(h, w, lab, dl, piece=512)
        dl[drop] = 0.0
        _verify(h, w, lab, dl, out)
        assert all(torch.equal(a, b) for a, b in zip(_run(h, w, lab, dl, piece=512), out))
    assert mfsdp.mfsdp_query_status() == 0


def test_bf16_tensor_core_large_logits_nan_and_dloss():
    h, w, lab, dl = _case(260, 264, 1100, "bf16", 0.0, seed=15, std=30.0)
    clean = _run(h, w, lab, dl)
    assert all(torch.isfinite(t).all() for t in clean)
    _verify(h, w, lab, dl, clean)
    _, _, dh, dw = _run(h, w, lab, torch.zeros_like(dl))
    assert not dh.any() and not dw.any()
    _, _, dh, dw = _run(h, w, lab, torch.full_like(dl, float("nan")))
    assert dh.isnan().all() and dw.isnan().all()
    h[17, 3] = float("nan")
    loss, lse, dh, _ = _run(h, w, lab, dl)
    keep = torch.arange(260, device="cuda") != 17
    assert loss[17].isnan() and lse[17].isnan() and dh[17].isnan().all()
    assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(dh[keep], clean[2][keep])


def test_nan_stays_in_its_token():
    h, w, lab, dl = _case(300, 64, 500, "bf16", 0.0, seed=6)
    clean = _run(h, w, lab, dl)
    h[17, 3] = float("nan")
    loss, lse, dh, _ = _run(h, w, lab, dl)
    keep = torch.arange(300, device="cuda") != 17
    assert loss[17].isnan() and lse[17].isnan() and dh[17].isnan().all()
    assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(dh[keep], clean[2][keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 300])
def test_dloss_of_zeros_and_of_nan(dtype, n):
    h, w, lab, dl = _case(n, 64, 500, dtype, 0.0, seed=13)
    _, _, dh, dw = _run(h, w, lab, torch.zeros_like(dl))
    assert not dh.any() and not dw.any()
    # a loss that overflowed upstream: no gradient may look like a valid one
    _, _, dh, dw = _run(h, w, lab, torch.full_like(dl, float("nan")))
    assert dh.isnan().all() and dw.isnan().all()
    _, _, dh, dw = _run(h, w, lab, torch.full_like(dl, float("inf")))
    assert not torch.isfinite(dh).any() and not torch.isfinite(dw).any()
    # one of them: its own row of dH, and dW
    if n > 1:
        clean = _run(h, w, lab, dl)[2]
        dl[17] = float("nan")
        _, _, dh, dw = _run(h, w, lab, dl)
        keep = torch.arange(n, device="cuda") != 17
        assert dh[17].isnan().all() and dw.isnan().all() and torch.isfinite(dh[keep]).all()
        assert ((dh[keep].float() - clean[keep].float()).abs()
                <= 2.0 ** -5 * clean[keep].float().abs().max()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_logits(dtype):
    # exp of the raw logits overflows and underflows: thousands on either side
    h, w, lab, dl = _case(260, 64, 800, dtype, 0.0, seed=7, std=60.0)
    out = _run(h, w, lab, dl)
    assert all(torch.isfinite(t).all() for t in out)
    _verify(h, w, lab, dl, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_gradient_alone_and_repeatable(dtype):
    from matrix_optimizer_owner_gb300 import mfsdp
    h, w, lab, dl = _case(310, 192, 1500, dtype, seed=8)
    loss, lse, dh, dw = _run(h, w, lab, dl, piece=512)
    for _ in range(2):
        again = _run(h, w, lab, dl, piece=512)
        assert all(torch.equal(a, b) for a, b in zip(again, (loss, lse, dh, dw)))
    assert torch.equal(_run(h, w, lab, dl, piece=512, want="h")[2], dh)
    assert torch.equal(_run(h, w, lab, dl, piece=512, want="w")[3], dw)
    mfsdp.mfsdp_head_loss_backward(h, w, lab, lse, dl, piece=512)      # neither: no work
    only = torch.empty_like(loss)
    mfsdp.mfsdp_head_loss_forward(h, w, lab, only, None)
    assert torch.equal(only, loss)
    inplace = h.clone()
    mfsdp.mfsdp_head_loss_backward(inplace, w, lab, lse, dl, inplace, piece=512)
    assert torch.equal(inplace, dh)


def test_no_tokens():
    from matrix_optimizer_owner_gb300 import mfsdp
    w = torch.randn(300, 48, device="cuda").bfloat16()
    h = torch.empty(0, 48, dtype=torch.bfloat16, device="cuda")
    lab, f = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    dw = torch.full_like(w, 5.0)
    mfsdp.mfsdp_head_loss_forward(h, w, lab, f, f)
    mfsdp.mfsdp_head_loss_backward(h, w, lab, f, f, h, dw)
    assert not dw.any()


def test_gradient_against_differences():
    """<dH, v> and <dW, v> against central differences of L = sum dloss loss in fp32, extrapolated
    from steps s and s / 2.  The extrapolation's error is below the difference of the quotients;
    the loss's rounding (the tolerance of the forward test) enters each quotient over 2 s."""
    h, w, lab, dl = _case(20, 40, 300, "f32", 0.2, seed=9)
    from matrix_optimizer_owner_gb300 import mfsdp
    _, _, dh, dw = _run(h, w, lab, dl)
    gen = torch.Generator(device="cuda").manual_seed(10)

    def total(hh, ww):
        loss = torch.empty(20, device="cuda")
        mfsdp.mfsdp_head_loss_forward(hh, ww, lab, loss, None)
        return float((loss.double() * dl.double()).sum())

    S = (np.abs(_np(h)) @ np.abs(_np(w)).T).max(axis=1)
    per_loss = 2 * (2 * _acc(40, "f32") * S + 2.0 ** -17 * (1 + S))
    noise = float((per_loss * np.abs(_np(dl))).sum())
    for base, grad, f in ((h, dh, lambda x: total(x, w)), (w, dw, lambda x: total(h, x))):
        v = torch.randn(base.shape, generator=gen, device="cuda")
        quot = [(f(base + s * v) - f(base - s * v)) / (2 * s) for s in (2.0 ** -4, 2.0 ** -5)]
        want = (4 * quot[1] - quot[0]) / 3
        got = float((grad.double() * v.double()).sum())
        assert abs(got - want) <= abs(quot[1] - quot[0]) + 3 * noise * 2 ** 5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_stream_and_graph(dtype):
    from matrix_optimizer_owner_gb300 import mfsdp
    h, w, lab, dl = _case(270, 128, 1100, dtype, seed=11)
    want = _run(h, w, lab, dl, piece=512)
    out = [torch.zeros_like(t) for t in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mfsdp.mfsdp_head_loss_forward(h, w, lab, out[0], out[1], stream=s)
    mfsdp.mfsdp_head_loss_backward(h, w, lab, out[1], dl, out[2], out[3], piece=512, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    ws = [torch.empty(mfsdp.mfsdp_head_loss_workspace_bytes(270, 128, w, back, 512 if back else 0),
                      dtype=torch.uint8, device="cuda") for back in (False, True)]
    for t in out:
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mfsdp.mfsdp_head_loss_forward(h, w, lab, out[0], out[1], workspace=ws[0])
        mfsdp.mfsdp_head_loss_backward(h, w, lab, out[1], dl, out[2], out[3], piece=512,
                                       workspace=ws[1])
    for _ in range(2):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert mfsdp.mfsdp_query_status() == 0


@pytest.mark.parametrize("vocab,piece,pitch", [(8192, 0, 0), (8192, 2048, 0), (8001, 1024, 8),
                                               (5000, 256, 3)])
def test_common_part_of_the_weight_stays_out_of_dhidden(vocab, piece, pitch):
    """W's rows share a part c, 20 times their spread.  A row of G sums to zero, so c cancels in dH =
    G W, and an error dG of G (its rounding to bf16 among them) must not meet it:
        |dH - ref| <= dG |W - c| + dG d + acc(V) |G| |W| + 2^-20 |G| |c| + 2^-8 |ref|
    with dG as in this file's head, d = 5 / sqrt(128) of W's spread for a c estimated from some 128
    rows, and the tensor cores' sum over V.  Labels are confident, so that G's largest entry is
    rounded too."""
    n, dim = 256, 64
    gen = torch.Generator(device="cuda").manual_seed(vocab + piece)
    spread = 2.0 / dim ** 0.5
    rows = torch.randn(vocab, dim, generator=gen, device="cuda") * spread
    common = torch.randn(dim, generator=gen, device="cuda") * 20 * spread
    w = _mat(vocab, dim, "bf16", gen, 1.0, pitch)
    w.copy_(rows + common)
    lab = torch.randint(vocab, (n,), generator=gen, device="cuda")
    h = (torch.randn(n, dim, generator=gen, device="cuda") + 0.6 / spread * rows[lab]).bfloat16()
    dl = torch.ones(n, device="cuda")
    dh = torch.empty_like(h)
    _, _, dh, _ = _run(h, w, lab, dl, piece=piece, dh=dh)
    H, W, L = _np(h), _np(w), lab.cpu().numpy()
    _, lse = oracle.forward(H, W, L)
    z = H @ W.T
    dz = _acc(dim, "bf16") * (np.abs(H) @ np.abs(W).T)
    dlse = dz.max(axis=1) + 2.0 ** -18 * (1 + np.abs(lse))
    _, G = oracle.logit_gradient(H, W, L, _np(dl))
    p = np.exp(z - lse[:, None])
    assert 0.2 < p[np.arange(n), L].mean() < 0.9
    rel = 2 * (dz.max(axis=1) + dlse)[:, None] + 2.0 ** -19 * (1 + np.abs(z) + np.abs(lse)[:, None])
    dG = p * rel + np.abs(G) * 2.0 ** -8
    ref, _ = oracle.backward(H, W, L, _np(dl))
    c = W.mean(axis=0)
    aG = np.abs(G) + dG
    tol = dG @ (np.abs(W - c) + 5 / 128 ** 0.5 * W.std(axis=0)) + _acc(vocab, "bf16") * (aG @ np.abs(W))
    tol += 2.0 ** -20 * aG.sum(axis=1, keepdims=True) * np.abs(c) + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(_np(dh) - ref) <= tol).all()


# one and two tokens on the tensor cores: widths between 256 and 1024 with large weights
@pytest.mark.parametrize("n,dim,vocab", [(1, 640, 60000), (2, 768, 80000), (1, 960, 40001)])
def test_few_tokens_backward_on_the_tensor_cores(n, dim, vocab):
    h, w, lab, dl = _case(n, dim, vocab, "bf16", 0.0, seed=n + dim)
    out = _run(h, w, lab, dl)
    _verify(h, w, lab, dl, out)
    assert all(torch.equal(a, b) for a, b in zip(_run(h, w, lab, dl), out))
