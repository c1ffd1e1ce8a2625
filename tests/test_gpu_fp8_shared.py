"""Inputs of the 8-bit operators that share a buffer, which only results may not."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _bytes(m):
    return m.data.view(torch.uint8), m.scales.view(torch.uint8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gate_and_up_of_one_checkpoint(dtype):
    """SwiGLU of one tensor with itself, from one checkpoint, as from two copies of it."""
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(0)
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    x, dy = (torch.randn(300, 520, generator=gen, device="cuda").to(t) for _ in range(2))
    one, two = mfsdp.fp8_empty(300, 520, 0), mfsdp.fp8_empty(300, 520, 0)
    for m in (one, two):
        mfsdp.mfsdp_quantize_fp8(x, m)
    got, want = [], []
    for outs, up in ((got, one), (want, two)):
        dg, du, col = torch.empty_like(dy), torch.empty_like(dy), mfsdp.fp8_empty(300, 520, 1)
        mfsdp.mfsdp_activation_backward(mfsdp.ACT_SWIGLU, dy, one, up, dg, du, dup8_col=col)
        outs += [dg, du, *_bytes(col)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_product_of_a_matrix_with_itself():
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(300, 520, generator=gen, device="cuda")
    a, b = mfsdp.fp8_empty(300, 520, 0), mfsdp.fp8_empty(300, 520, 0)
    for m in (a, b):
        mfsdp.mfsdp_quantize_fp8(x, m)
    c, d = torch.empty(300, 300, device="cuda"), torch.empty(300, 300, device="cuda")
    mfsdp.mfsdp_gemm_fp8(a, a, c, trans_b=True)
    mfsdp.mfsdp_gemm_fp8(a, b, d, trans_b=True)
    assert torch.equal(c, d)
