"""The norm, embedding and head-loss operators on buffers of more than 2^31 elements: rows past that
offset come out as they do from small buffers."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_norm_rows_past_32_bit_offsets():
    from matrix_optimizer_owner_gb300 import mfsdp
    rows, cols, tail = 263000, 8192, 500            # 2.15e9 elements
    assert (rows - tail) * cols > 2 ** 31
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(0)
    x[-tail:] = torch.randn(tail, cols, generator=gen, device="cuda")
    dy = torch.zeros_like(x)
    dy[-tail:] = torch.randn(tail, cols, generator=gen, device="cuda")
    w = torch.randn(cols, generator=gen, device="cuda")

    def run(x, dy):
        n = x.shape[0]
        mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        dw = torch.empty(cols, device="cuda")
        y = torch.empty_like(x)
        mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x, w, None, 1e-5, y, mean, rstd)
        y_tail = y[-tail:].clone()
        mfsdp.mfsdp_norm_backward(mfsdp.NORM_LAYER, dy, x, w, mean, rstd, y, dw)
        return y_tail, y[-tail:].clone(), dw

    big, small = run(x, dy), run(x[-tail:].clone(), dy[-tail:].clone())
    assert torch.equal(big[0], small[0]) and torch.equal(big[1], small[1])
    # zero rows add nothing, but the rows fall to other blocks: the sums differ in order only
    bound = (tail + 64) * 2.0 ** -24 * (dy[-tail:].float().abs() *
                                        (x[-tail:].float().abs() + 1) * small[2].new_tensor(2.0)).sum(0)
    assert ((big[2] - small[2]).abs() <= 2 * bound).all()


def test_embedding_rows_past_32_bit_offsets():
    from matrix_optimizer_owner_gb300 import mfsdp
    vocab, dim, n = 2100100, 1024, 300
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = vocab - 1 - torch.randint(90, (n,), generator=gen, device="cuda")
    table[-90:] = torch.randn(90, dim, generator=gen, device="cuda")
    assert int(ids.min()) * dim > 2 ** 31
    out = torch.empty(n, dim, dtype=torch.bfloat16, device="cuda")
    mfsdp.mfsdp_embedding_forward(table, ids, 1.0, out)
    assert torch.equal(out, table[ids])
    table.fill_(7.0)
    mfsdp.mfsdp_embedding_backward(ids, out, 1.0, table)
    small = torch.empty(90, dim, dtype=torch.bfloat16, device="cuda")
    mfsdp.mfsdp_embedding_backward(ids - (vocab - 90), out, 1.0, small)
    assert torch.equal(table[-90:], small)
    assert not table[:-90].any()


@pytest.mark.parametrize("n", [2, 70])
def test_head_loss_rows_past_32_bit_offsets(n):
    """A weight that is zero but for its last rows: lse = log(zeros + sum exp(z)), and the gradient
    of a zero row is p hidden with p = exp(-lse)."""
    from matrix_optimizer_owner_gb300 import mfsdp
    vocab, dim, last = 2100100, 1024, 64
    gen = torch.Generator(device="cuda").manual_seed(n)
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    w[-last:] = torch.randn(last, dim, generator=gen, device="cuda") * 0.5
    assert (vocab - last) * dim > 2 ** 31
    h = torch.randn(n, dim, generator=gen, device="cuda").bfloat16()
    labels = vocab - 1 - torch.randint(last, (n,), generator=gen, device="cuda")
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    mfsdp.mfsdp_head_loss_forward(h, w, labels, loss, lse)
    z = h.double() @ w[-last:].double().T
    want = torch.logsumexp(torch.cat([z, torch.full((n, 1), math.log(vocab - last), device="cuda",
                                                    dtype=torch.float64)], 1), 1)
    at = z.gather(1, (labels - (vocab - last))[:, None])[:, 0]
    # the bounds of the head loss's own test: (K / 16 + 8) 2^-22 sum |h w| and 2^-18 (1 + |lse|)
    dz = ((dim / 16 + 8) * 2.0 ** -22 * (h.double().abs() @ w[-last:].double().abs().T)).max(1).values
    tol = dz + 2.0 ** -18 * (1 + want.abs())
    assert ((lse.double() - want).abs() <= tol).all()
    assert ((loss.double() - (want - at)).abs() <= 2 * tol).all()
    dl = torch.ones(n, device="cuda")
    dh, dw = torch.empty_like(h), torch.full_like(w, 3.0)
    mfsdp.mfsdp_head_loss_backward(h, w, labels, lse, dl, dh, dw)
    g = torch.softmax(torch.cat([z, z.new_full((n, 1), math.log(vocab - last))], 1), 1)[:, :last]
    g = g.scatter_add(1, (labels - (vocab - last))[:, None], -g.new_ones(n, 1))
    for got, ref, mag in ((dh, g @ w[-last:].double(), g.abs() @ w[-last:].double().abs()),
                          (dw[-last:], g.T @ h.double(), g.abs().T @ h.double().abs())):
        # 2^-8 for the entries of g, as much for the result, and the errors of the logits
        bound = mag * (2.0 ** -8 + 2 * float(tol.max())) + ref.abs() * 2.0 ** -8 + 1e-6 * mag
        assert ((got.double() - ref).abs() <= bound + 1e-12).all()
    zero = (torch.exp(-want)[:, None] * h.double()).sum(0)
    mag = (torch.exp(-want)[:, None] * h.double().abs()).sum(0)
    rows = dw[[0, 1, 1000000, vocab - last - 1]].double()
    assert ((rows - zero).abs() <= mag * (2.0 ** -8 + 2 * float(tol.max())) + zero.abs() * 2.0 ** -8).all()
