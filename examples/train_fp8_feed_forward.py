"""A residual feed-forward block trained in 8 bits on the library's kernels.

    h = x + r;  y = rms_norm(h);  z = swiglu(y Wg^T, y Wu^T);  out = h + z Wd^T

The operands of every product are held in 8 bits, and so is what the backward pass needs of the forward
pass: h, the two products and the operands y and z.  The three matrices are the Muon matrices of an owner
step; their gradients are written into its contribution buffer, and their 8-bit copies are made of its
fp32 master weights each step.  The norm's weight is the AdamW tail.  It is fitted to a fixed random block.

    python examples/train_fp8_feed_forward.py [--steps 60]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from matrix_optimizer_owner_gb300 import mfsdp  # noqa: E402
from matrix_optimizer_owner_gb300.mfsdp import GROUPS_COL, GROUPS_ROW, GROUPS_TILE  # noqa: E402
from matrix_optimizer_owner_gb300.owner_step import OwnerStep  # noqa: E402
from workloads.configs import Hyper  # noqa: E402


class FeedForward:
    """Parameters, optimizer state and gradients in an OwnerStep's flat buffers."""

    def __init__(self, dim: int, hidden: int, n_tokens: int, seed: int = 0, eps: float = 1e-5):
        self.dim, self.hidden, self.n, self.eps = dim, hidden, n_tokens, eps
        shapes = {"gate": (hidden, dim), "up": (hidden, dim), "down": (dim, hidden)}
        each = dim * hidden
        self.owner = OwnerStep(list(shapes.values()), [0, each, 2 * each], dim, device="cuda")
        self.grad = torch.zeros_like(self.owner.weights)
        self.norm_w, self.norm_grad = self.owner.tail_p, torch.zeros_like(self.owner.tail_p)
        self.w, self.g, self.w8 = {}, {}, {}
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for i, (name, (rows, cols)) in enumerate(shapes.items()):
            at = slice(i * each, (i + 1) * each)
            self.w[name] = self.owner.weights[at].view(rows, cols)
            self.g[name] = self.grad[at].view(rows, cols)
            self.w8[name] = mfsdp.fp8_empty(rows, cols, GROUPS_TILE)
            self.w[name].normal_(0.0, cols ** -0.5, generator=gen)
        self.norm_w.fill_(1.0)
        row = lambda cols, dtype=None: mfsdp.fp8_empty(n_tokens, cols, GROUPS_ROW, dtype)  # noqa: E731
        col = lambda cols, dtype=None: mfsdp.fp8_empty(n_tokens, cols, GROUPS_COL, dtype)  # noqa: E731
        bf = lambda cols: torch.empty(n_tokens, cols, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        e5 = torch.float8_e5m2
        # kept from the forward pass: 8 bits a value
        self.h8, self.y8, self.z8 = row(dim), row(dim), row(hidden)
        self.gate8, self.up8, self.rstd = row(hidden), row(hidden), torch.empty(n_tokens, device="cuda")
        # passing
        self.h, self.out, self.gate, self.up = bf(dim), bf(dim), bf(hidden), bf(hidden)
        self.dy, self.dz, self.dx = bf(dim), bf(hidden), bf(dim)
        self.dout8, self.dout8_col = row(dim, e5), col(dim, e5)
        self.dgate8, self.dgate8_col = row(hidden, e5), col(hidden, e5)
        self.dup8, self.dup8_col = row(hidden, e5), col(hidden, e5)
        self.y8_col, self.z8_col = col(dim), col(hidden)

    def forward(self, x, r):
        """The block's output for a branch ``x`` and the residual stream ``r`` (bfloat16)."""
        for name, w in self.w.items():
            mfsdp.mfsdp_quantize_fp8(w, self.w8[name])
        mfsdp.mfsdp_norm_residual_forward(mfsdp.NORM_RMS, x, r, self.norm_w, None, self.eps, h=self.h,
                                          y8=self.y8, h8=self.h8, rstd=self.rstd)
        mfsdp.mfsdp_gemm_fp8(self.y8, self.w8["gate"], self.gate, trans_b=True)
        mfsdp.mfsdp_gemm_fp8(self.y8, self.w8["up"], self.up, trans_b=True)
        mfsdp.mfsdp_activation_forward(mfsdp.ACT_SWIGLU, self.gate, self.up, y8=self.z8,
                                       gate8=self.gate8, up8=self.up8)
        self.out.copy_(self.h)
        mfsdp.mfsdp_gemm_fp8(self.z8, self.w8["down"], self.out, trans_b=True, accumulate=True)
        return self.out

    def backward(self, dout):
        """Every parameter's gradient, into ``grad`` and ``norm_grad``; the inputs' as the result."""
        mfsdp.mfsdp_quantize_fp8(dout, self.dout8, self.dout8_col)
        mfsdp.mfsdp_regroup_fp8(self.z8, self.z8_col)
        mfsdp.mfsdp_gemm_fp8(self.dout8_col, self.z8_col, self.g["down"], trans_a=True)
        mfsdp.mfsdp_gemm_fp8(self.dout8, self.w8["down"], self.dz)
        mfsdp.mfsdp_activation_backward(mfsdp.ACT_SWIGLU, self.dz, self.gate8, self.up8,
                                        dgate8=self.dgate8, dup8=self.dup8,
                                        dgate8_col=self.dgate8_col, dup8_col=self.dup8_col)
        mfsdp.mfsdp_regroup_fp8(self.y8, self.y8_col)
        mfsdp.mfsdp_gemm_fp8(self.dgate8_col, self.y8_col, self.g["gate"], trans_a=True)
        mfsdp.mfsdp_gemm_fp8(self.dup8_col, self.y8_col, self.g["up"], trans_a=True)
        mfsdp.mfsdp_gemm_fp8(self.dgate8, self.w8["gate"], self.dy)
        mfsdp.mfsdp_gemm_fp8(self.dup8, self.w8["up"], self.dy, accumulate=True)
        mfsdp.mfsdp_norm_residual_backward(mfsdp.NORM_RMS, self.dy, dout, self.h8, self.norm_w, None,
                                           self.rstd, self.dx, self.norm_grad)
        return self.dx

    def step(self, hyper: Hyper):
        self.owner.step([self.grad], [self.norm_grad], hyper)


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=640)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    model = FeedForward(a.dim, a.hidden, a.tokens)
    teacher = FeedForward(a.dim, a.hidden, a.tokens, seed=7)
    hyper = Hyper(lr=0.02, weight_decay=0.0, adam_lr=3e-3, adam_wd=0.0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for t in range(a.steps):
        x, r = (torch.randn(a.tokens, a.dim, generator=gen, device="cuda").bfloat16() for _ in range(2))
        diff = model.forward(x, r).float() - teacher.forward(x, r).float()
        model.backward((diff / a.tokens).bfloat16())
        model.step(hyper)
        if t % 10 == 0 or t == a.steps - 1:
            print(f"step {t:4d}  loss {float(diff.square().mean()):.4f}")
    assert mfsdp.mfsdp_query_status() == 0


if __name__ == "__main__":
    main()
