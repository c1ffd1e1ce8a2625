"""A small language model trained end to end on the library's kernels.

    x = embedding[tokens];  n = layer_norm(x);  h = n W^T;  y = rms_norm(h)
    loss = mean over the labelled tokens of the cross entropy of y embedding^T

The embedding and the head are one fp32 table.  W is the Muon matrix of an owner step; the table
and the norms' vectors are its packed AdamW tail, one flat buffer, and the operators write their
gradients straight into the tail's contribution: the head's gradient overwrites the table's slot
and the lookup's gradient is added to it.

    python examples/train_tied_lm.py [--steps 100]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from matrix_optimizer_owner_gb300 import mfsdp  # noqa: E402
from matrix_optimizer_owner_gb300.owner_step import OwnerStep  # noqa: E402
from workloads.configs import Hyper  # noqa: E402

IGNORE = -100


class TiedLM:
    """Parameters, optimizer state and gradients in an OwnerStep's flat buffers."""

    def __init__(self, vocab: int, dim: int, n_tokens: int, seed: int = 0, eps: float = 1e-5):
        self.vocab, self.dim, self.n, self.eps = vocab, dim, n_tokens, eps
        sizes = {"table": vocab * dim, "ln_w": dim, "ln_b": dim, "rms_w": dim}
        self.owner = OwnerStep([(dim, dim)], [0], sum(sizes.values()), device="cuda")
        self.tail_grad = torch.zeros_like(self.owner.tail_p)
        self.p, self.g, at = {}, {}, 0
        for name, size in sizes.items():
            self.p[name] = self.owner.tail_p[at:at + size]
            self.g[name] = self.tail_grad[at:at + size]
            at += size
        for d in (self.p, self.g):
            d["table"] = d["table"].view(vocab, dim)
        self.w = self.owner.weights[:dim * dim].view(dim, dim)
        self.w_grad = torch.zeros_like(self.w)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.p["table"].normal_(0.0, 0.05, generator=gen)
        self.p["ln_w"].fill_(1.0)
        self.p["rms_w"].fill_(1.0)
        self.w.normal_(0.0, dim ** -0.5, generator=gen)
        new = lambda *shape: torch.empty(shape, device="cuda")  # noqa: E731
        self.x, self.norm, self.h, self.y = (new(n_tokens, dim) for _ in range(4))
        self.dy, self.dh, self.dnorm, self.dx = (new(n_tokens, dim) for _ in range(4))
        self.mean, self.rstd, self.rstd2, self.loss, self.lse = (new(n_tokens) for _ in range(5))

    def forward(self, tokens, labels):
        """Loss per token (0 where the label is IGNORE)."""
        mfsdp.mfsdp_embedding_forward(self.p["table"], tokens, 1.0, self.x)
        mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, self.x, self.p["ln_w"], self.p["ln_b"],
                                 self.eps, self.norm, self.mean, self.rstd)
        mfsdp.mfsdp_gemm_f32_batched([(self.norm, self.w, self.h, 1.0, 0.0)], trans_b=True)
        mfsdp.mfsdp_norm_forward(mfsdp.NORM_RMS, self.h, self.p["rms_w"], None, self.eps, self.y,
                                 None, self.rstd2)
        mfsdp.mfsdp_head_loss_forward(self.y, self.p["table"], labels, self.loss, self.lse,
                                      ignore_index=IGNORE)
        return self.loss

    def backward(self, tokens, labels, dloss):
        """Every parameter's gradient, into ``tail_grad`` and ``w_grad``."""
        mfsdp.mfsdp_head_loss_backward(self.y, self.p["table"], labels, self.lse, dloss, self.dy,
                                       self.g["table"], ignore_index=IGNORE)
        mfsdp.mfsdp_norm_backward(mfsdp.NORM_RMS, self.dy, self.h, self.p["rms_w"], None,
                                  self.rstd2, self.dh, self.g["rms_w"])
        mfsdp.mfsdp_gemm_f32_batched([(self.dh, self.norm, self.w_grad, 1.0, 0.0)], trans_a=True)
        mfsdp.mfsdp_gemm_f32_batched([(self.dh, self.w, self.dnorm, 1.0, 0.0)])
        mfsdp.mfsdp_norm_backward(mfsdp.NORM_LAYER, self.dnorm, self.x, self.p["ln_w"], self.mean,
                                  self.rstd, self.dx, self.g["ln_w"], self.g["ln_b"])
        mfsdp.mfsdp_embedding_backward(tokens, self.dx, 1.0, self.g["table"], accumulate=True)

    def step(self, tokens, labels, hyper: Hyper):
        """One training step; the loss per token before it."""
        loss = self.forward(tokens, labels)
        live = (labels != IGNORE).sum()
        self.backward(tokens, labels, (1.0 / live).expand(self.n).contiguous())
        self.owner.step([self.w_grad.view(-1)], [self.tail_grad], hyper)
        return loss


def batch(vocab: int, n: int, gen):
    """Tokens whose successor is a fixed permutation of them, every 16th label left out."""
    tokens = torch.randint(vocab, (n,), generator=gen, device="cuda")
    labels = (tokens * 7 + 3) % vocab
    labels[::16] = IGNORE
    return tokens, labels


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    model = TiedLM(a.vocab, a.dim, a.tokens)
    hyper = Hyper(lr=0.02, weight_decay=0.0, adam_lr=3e-3, adam_wd=0.0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for t in range(a.steps):
        tokens, labels = batch(a.vocab, a.tokens, gen)
        loss = model.step(tokens, labels, hyper)
        if t % 10 == 0 or t == a.steps - 1:
            live = int((labels != IGNORE).sum())
            print(f"step {t:4d}  loss {float(loss.sum()) / live:.4f}")
    assert mfsdp.mfsdp_query_status() == 0


if __name__ == "__main__":
    main()
