"""The operators as one training step (examples/train_tied_lm.py): every gradient of the model,
the tied table's two parts included, against 64-bit automatic differentiation; and training.

Tolerance: each gradient is a chain of fp32 operators whose products keep about 20 bits
(3xTF32: 2^-20 per product), through two norms and a softmax.  Relative to the gradient's norm the
first-order error is below the number of operators it passes (7) times 2^-18, the same bound per
operator that the head loss's test derives for its products: 3e-5."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "train_tied_lm", os.path.join(ROOT, "examples", "train_tied_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_of_a_step():
    ex = _example()
    m = ex.TiedLM(500, 96, 300, seed=3)
    for name in ("ln_w", "ln_b", "rms_w"):
        m.p[name].add_(torch.randn(96, device="cuda") * 0.1)
    tokens, labels = ex.batch(500, 300, torch.Generator(device="cuda").manual_seed(4))
    live = (labels != ex.IGNORE)
    dloss = torch.full((300,), 1.0 / int(live.sum()), device="cuda")
    loss = m.forward(tokens, labels).clone()
    m.backward(tokens, labels, dloss)
    P = {k: v.detach().double().requires_grad_() for k, v in m.p.items()}
    W = m.w.detach().double().requires_grad_()
    x = P["table"][tokens]
    mu, var = x.mean(1, keepdim=True), x.var(1, keepdim=True, unbiased=False)
    n = (x - mu) / torch.sqrt(var + m.eps) * P["ln_w"] + P["ln_b"]
    h = n @ W.T
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + m.eps) * P["rms_w"]
    z = y @ P["table"].T
    ref = torch.logsumexp(z, 1) - z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    (ref[live].sum() / int(live.sum())).backward()
    assert torch.allclose(loss[live].double(), ref[live], rtol=3e-5, atol=3e-5)
    assert not loss[~live].any()
    for name, grad in [(k, m.g[k]) for k in P] + [("w", m.w_grad)]:
        want = (W if name == "w" else P[name]).grad
        assert (grad.double() - want).norm() <= 3e-5 * want.norm(), name


def test_training_lowers_the_loss():
    ex = _example()
    m = ex.TiedLM(200, 128, 1024, seed=5)
    hyper = ex.Hyper(lr=0.02, weight_decay=0.0, adam_lr=3e-3, adam_wd=0.0)
    gen = torch.Generator(device="cuda").manual_seed(6)
    means = []
    for _ in range(60):
        tokens, labels = ex.batch(200, 1024, gen)
        loss = m.step(tokens, labels, hyper)
        means.append(float(loss.sum()) / int((labels != ex.IGNORE).sum()))
    # the task is a permutation of the tokens: from ln 200 = 5.3 towards 0
    assert 4.0 < means[0] < 8.0 and means[-1] < 0.5 * means[0]
    assert ex.mfsdp.mfsdp_query_status() == 0
