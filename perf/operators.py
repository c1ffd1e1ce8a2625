"""The operators of a language model's first, last and normalisation parameters, as measured cases.

The owner step (``matrix_optimizer_owner_gb300.owner_step``) consumes gradients: matrices go to
Muon, and vectors, embeddings and the output head go to AdamW.  The operators here are the ones
whose weights live in that AdamW share, and which produce its gradients:

``norm``       layer norm and RMS norm, forward, and backward with the reduction of the weight's
               and the bias's gradient over the rows;
``embedding``  the lookup with a scale, and the gradient of the table, summed over the tokens of
               each id;
``head_loss``  softmax cross entropy of ``hidden @ weight.T`` per token, in pieces of the
               vocabulary and without keeping the logits, and its gradient for both factors.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once
at the end) or, where ``own`` is true, through the public entry points of the library.
"""

from __future__ import annotations

import math
import random

import torch

own = False

IGNORE = -100
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INDEX = {"i64": torch.int64, "i32": torch.int32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One token through one layer norm of the GPT-2-small width: a decoding step's smallest
        # call, where only latency counts.
        dict(name="norm_forward_one_row", op="norm", kind="layer", train=False, rows=1, cols=768,
             dtype="bf16", params="f32"),
        # A GPT-2-small training step's norm: 16 sequences of 1024 tokens, fp32 tail parameters.
        dict(name="norm_train_768", op="norm", kind="layer", train=True, rows=16384, cols=768,
             dtype="bf16", params="f32"),
        # A Llama-3-8B training step's RMS norm.
        dict(name="norm_train_rms_4096", op="norm", kind="rms", train=True, rows=8192, cols=4096,
             dtype="bf16", params="bf16"),
        # An odd width in fp32: no row but the first starts on a vector boundary.
        dict(name="norm_train_f32_odd", op="norm", kind="layer", train=True, rows=1023,
             cols=1001, dtype="f32", params="f32"),
        # The lookup of a training step from the fp32 master table into bf16 activations.
        dict(name="embedding_forward_768", op="embedding", train=False, tokens=16384, dim=768,
             vocab=50257, table="f32", dtype="bf16", index="i64", zipf=True, scale=1.0,
             padding=-1),
        # Its gradient over the GPT-2 vocabulary; token frequencies fall off as in text, so one
        # id owns a few per cent of the tokens and most rows of the gradient are zero.
        dict(name="embedding_grad_768", op="embedding", train=True, tokens=16384, dim=768,
             vocab=50257, table="bf16", dtype="bf16", index="i64", zipf=True, scale=1.0,
             padding=-1),
        # The same for a large table, with the sqrt(dim) scale some models put on the lookup.
        dict(name="embedding_grad_4096", op="embedding", train=True, tokens=8192, dim=4096,
             vocab=128256, table="bf16", dtype="bf16", index="i32", zipf=True, scale=64.0,
             padding=-1),
        # A small odd table in fp32 with a padding id that takes no gradient.
        dict(name="embedding_grad_f32_odd", op="embedding", train=True, tokens=1001, dim=301,
             vocab=5003, table="f32", dtype="f32", index="i64", zipf=False, scale=1.0,
             padding=0),
        # Scoring one token against the GPT-2 vocabulary: the smallest evaluation call, one
        # pass over the head's weight.
        dict(name="head_loss_eval_one_token", op="head_loss", train=False, tokens=1, dim=768,
             vocab=50257, dtype="bf16", index="i64", ignored=0.0),
        # A GPT-2-small training step's head: loss, lse and both gradients.
        dict(name="head_loss_train_768", op="head_loss", train=True, tokens=8192, dim=768,
             vocab=50257, dtype="bf16", index="i64", ignored=0.0),
        # A large head in instruction tuning: a quarter of the tokens (the prompts) carry the
        # ignored label and take no part.
        dict(name="head_loss_train_4096", op="head_loss", train=True, tokens=4096, dim=4096,
             vocab=128256, dtype="bf16", index="i64", ignored=0.25),
        # Odd sizes in fp32, as a test or a small fp32 model has them.
        dict(name="head_loss_train_f32_odd", op="head_loss", train=True, tokens=333, dim=100,
             vocab=1031, dtype="f32", index="i32", ignored=0.1),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range: as often a multiple of 64 as not."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 64:
        n -= n % 64
    return max(lo, min(hi, n))


def draw(rng: random.Random):
    op = rng.choice(["norm", "embedding", "head_loss"])
    if op == "norm":
        return dict(op=op, kind=rng.choice(["layer", "rms"]), train=rng.random() < 0.7,
                    rows=_size(rng, 1, 32768), cols=_size(rng, 64, 8192),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), params=rng.choice(["f32", "bf16"]))
    if op == "embedding":
        train = rng.random() < 0.7
        dtype = rng.choice(["bf16", "bf16", "f32"])
        vocab = _size(rng, 1000, 128256)
        return dict(op=op, train=train, tokens=_size(rng, 1, 32768), dim=_size(rng, 64, 4096),
                    vocab=vocab, table=rng.choice(["bf16", "f32"]), dtype=dtype,
                    index=rng.choice(["i64", "i32"]), zipf=rng.random() < 0.7,
                    scale=rng.choice([1.0, 8.0]),
                    padding=rng.choice([-1, rng.randrange(vocab)]))
    return dict(op=op, train=rng.random() < 0.7, tokens=_size(rng, 1, 4096),
                dim=_size(rng, 64, 4096), vocab=_size(rng, 1000, 128256),
                dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
                index=rng.choice(["i64", "i32"]), ignored=rng.choice([0.0, 0.0, 0.1, 0.5]))


# ------------------------------------------------------------------------------------ inputs
def _ids(case, gen, n):
    """Token ids: uniform, or with the frequencies of text (Zipf's law over shuffled ids)."""
    v = case["vocab"]
    if case.get("zipf", True):
        rank = torch.arange(v, device="cuda", dtype=torch.float64)
        cdf = torch.cumsum(1.0 / (rank + 2.7), 0)
        u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64) * cdf[-1]
        shuffle = torch.randperm(v, generator=gen, device="cuda")
        ids = shuffle[torch.searchsorted(cdf, u).clamp_(max=v - 1)]
    else:
        ids = torch.randint(v, (n,), generator=gen, device="cuda")
    return ids.to(INDEX[case["index"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype="f32", mean=0.0):
        t = torch.randn(shape, generator=gen, device="cuda").mul_(std)
        return (t.add_(mean) if mean else t).to(DTYPES[dtype])

    def out(*shape, dtype="f32"):
        return torch.empty(shape, dtype=DTYPES[dtype], device="cuda")

    s = dict(case)
    if case["op"] == "norm":
        r, c, d, p = case["rows"], case["cols"], case["dtype"], case["params"]
        # a residual stream: rows of different scale, off centre
        x = normal(r, c) * normal(r, 1, std=0.5).exp() + normal(r, 1, std=0.3)
        s.update(x=x.to(DTYPES[d]), weight=normal(c, std=0.1, mean=1.0, dtype=p),
                 bias=normal(c, std=0.1, dtype=p) if case["kind"] == "layer" else None,
                 y=out(r, c, dtype=d), mean=out(r) if case["kind"] == "layer" else None,
                 rstd=out(r))
        if case["train"]:
            s.update(dy=normal(r, c, std=1e-3, dtype=d), dx=out(r, c, dtype=d),
                     dweight=out(c, dtype=p),
                     dbias=out(c, dtype=p) if case["kind"] == "layer" else None)
        return s
    if case["op"] == "embedding":
        n, c, d = case["tokens"], case["dim"], case["dtype"]
        s.update(ids=_ids(case, gen, n))
        if case["train"]:
            s.update(dy=normal(n, c, std=1e-3, dtype=d),
                     dtable=out(case["vocab"], c, dtype=case["table"]))
        else:
            s.update(weight=normal(case["vocab"], c, std=0.02, dtype=case["table"]),
                     out=out(n, c, dtype=d))
        return s
    n, c, v, d = case["tokens"], case["dim"], case["vocab"], case["dtype"]
    labels = _ids(case, gen, n)
    drop = torch.randperm(n, generator=gen, device="cuda")[:_ignored(case)]
    labels[drop] = IGNORE
    # normalised activations against weights that give logits of a trained model's spread
    s.update(hidden=normal(n, c, dtype=d), weight=normal(v, c, std=2.0 / math.sqrt(c), dtype=d),
             labels=labels, loss=out(n), lse=out(n))
    if case["train"]:
        s.update(dloss=torch.full((n,), 1.0 / max(n - _ignored(case), 1), device="cuda"),
                 dhidden=out(n, c, dtype=d), dweight=out(v, c, dtype=d))
    return s


def _ignored(case):
    return int(case["tokens"] * case["ignored"])


# ------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _RUN_OWN[state["op"]](state)
    with torch.no_grad():
        return _RUN_PLAIN[state["op"]](state)


def _plain_norm(s):
    x, w = s["x"].float(), s["weight"].float()
    layer = s["kind"] == "layer"
    mean = x.mean(1) if layer else None
    xc = x - mean[:, None] if layer else x
    rstd = ((xc * xc).mean(1) + EPS).rsqrt()
    xh = xc * rstd[:, None]
    y = xh * w
    if layer:
        y = y + s["bias"].float()
    res = {"y": y.to(s["x"].dtype), "rstd": rstd}
    if layer:
        res["mean"] = mean
    if s["train"]:
        dy = s["dy"].float()
        g = dy * w
        dx = g - xh * (g * xh).mean(1, keepdim=True)
        if layer:
            dx = dx - g.mean(1, keepdim=True)
            res["dbias"] = dy.sum(0).to(s["weight"].dtype)
        res["dx"] = (dx * rstd[:, None]).to(s["x"].dtype)
        res["dweight"] = (dy * xh).sum(0).to(s["weight"].dtype)
    return res


def _plain_embedding(s):
    ids = s["ids"].long()
    if not s["train"]:
        return (s["weight"][ids].float() * s["scale"]).to(s["out"].dtype)
    dy = s["dy"].float() * s["scale"]
    if s["padding"] >= 0:
        dy = dy * (ids != s["padding"])[:, None]
    grad = torch.zeros(s["dtable"].shape, device=dy.device).index_add_(0, ids, dy)
    return grad.to(s["dtable"].dtype)


def _plain_head_loss(s):
    h, w = s["hidden"].float(), s["weight"].float()
    keep = s["labels"] != IGNORE
    lab = torch.where(keep, s["labels"], 0).long()[:, None]
    logits = h @ w.T
    top = logits.max(1, keepdim=True).values
    at = logits.gather(1, lab)
    p = (logits - top).exp()
    del logits
    total = p.sum(1, keepdim=True)
    lse = top + total.log()
    zero = torch.zeros((), device=h.device)
    res = {"loss": torch.where(keep, (lse - at)[:, 0], zero),
           "lse": torch.where(keep, lse[:, 0], zero)}
    if s["train"]:
        g = torch.where(keep, s["dloss"], zero)[:, None]
        p.mul_(g / total).scatter_add_(1, lab, -g)
        res["dhidden"] = (p @ w).to(s["hidden"].dtype)
        res["dweight"] = (p.T @ h).to(s["weight"].dtype)
    return res


def _own_norm(s):
    from matrix_optimizer_owner_gb300 import mfsdp
    kind = mfsdp.NORM_LAYER if s["kind"] == "layer" else mfsdp.NORM_RMS
    mfsdp.mfsdp_norm_forward(kind, s["x"], s["weight"], s["bias"], EPS, s["y"], s["mean"],
                             s["rstd"])
    names = ["y", "rstd"] + (["mean"] if s["kind"] == "layer" else [])
    if s["train"]:
        mfsdp.mfsdp_norm_backward(kind, s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                                  s["dx"], s["dweight"], s["dbias"])
        names += (["dbias"] if s["kind"] == "layer" else []) + ["dx", "dweight"]
    return {k: s[k] for k in names}


def _own_embedding(s):
    from matrix_optimizer_owner_gb300 import mfsdp
    if not s["train"]:
        mfsdp.mfsdp_embedding_forward(s["weight"], s["ids"], s["scale"], s["out"])
        return s["out"]
    mfsdp.mfsdp_embedding_backward(s["ids"], s["dy"], s["scale"], s["dtable"],
                                   padding_idx=s["padding"])
    return s["dtable"]


def _own_head_loss(s):
    from matrix_optimizer_owner_gb300 import mfsdp
    mfsdp.mfsdp_head_loss_forward(s["hidden"], s["weight"], s["labels"], s["loss"], s["lse"],
                                  ignore_index=IGNORE)
    names = ["loss", "lse"]
    if s["train"]:
        mfsdp.mfsdp_head_loss_backward(s["hidden"], s["weight"], s["labels"], s["lse"],
                                       s["dloss"], s["dhidden"], s["dweight"],
                                       ignore_index=IGNORE)
        names += ["dhidden", "dweight"]
    return {k: s[k] for k in names}


_RUN_PLAIN = {"norm": _plain_norm, "embedding": _plain_embedding, "head_loss": _plain_head_loss}
_RUN_OWN = {"norm": _own_norm, "embedding": _own_embedding, "head_loss": _own_head_loss}


# ------------------------------------------------------------------------------------ work
def work(case):
    if case["op"] == "norm":
        r, c, layer = case["rows"], case["cols"], case["kind"] == "layer"
        e, p = r * c * BYTES[case["dtype"]], c * BYTES[case["params"]] * (2 if layer else 1)
        stats = r * 4 * (2 if layer else 1)
        if not case["train"]:
            return {"bytes": 2 * e + p + stats, "flops": 6 * r * c}
        # x, dy in; y, dx and the parameters' gradients out
        return {"bytes": 4 * e + 2 * p + stats, "flops": 18 * r * c}
    if case["op"] == "embedding":
        n, c, v = case["tokens"], case["dim"], case["vocab"]
        ids = n * (8 if case["index"] == "i64" else 4)
        act = n * c * BYTES[case["dtype"]]
        if case["train"]:
            return {"bytes": ids + act + v * c * BYTES[case["table"]], "flops": 2 * n * c}
        # each table row that is looked up is read once: the expected number of distinct ids
        p = 1.0 / (torch.arange(v, dtype=torch.float64) + 2.7) if case["zipf"] else torch.ones(v)
        rows = float((1.0 - (1.0 - p.double() / p.sum()) ** n).sum())
        return {"bytes": int(ids + act + rows * c * BYTES[case["table"]]), "flops": n * c}
    n, c, v = case["tokens"], case["dim"], case["vocab"]
    b, live = BYTES[case["dtype"]], case["tokens"] - _ignored(case)
    ids = n * (8 if case["index"] == "i64" else 4)
    if not case["train"]:
        return {"bytes": (live + v) * c * b + ids + 8 * n, "flops": 2 * live * c * v}
    # one product for the logits and one for each gradient
    return {"bytes": 2 * (n + v) * c * b + ids + 12 * n, "flops": 6 * live * c * v}


# ------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """What ``run`` returns, from the definitions in 64 bits."""
    with torch.no_grad():
        return _EXACT[case["op"]](prepare(case, seed))


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    layer = s["kind"] == "layer"
    n = x.shape[1]
    mu = x.sum(1) / n if layer else torch.zeros_like(x[:, 0])
    var = ((x - mu[:, None]) ** 2).sum(1) / n
    sigma = torch.sqrt(var + EPS)
    z = (x - mu[:, None]) / sigma[:, None]
    res = {"y": z * w + s["bias"].double() if layer else z * w, "rstd": 1 / sigma}
    if layer:
        res["mean"] = mu
    if s["train"]:
        dy = s["dy"].double()
        dz = dy * w
        # d/dx of z = (x - mu(x)) / sigma(x): the projection off z and, for a layer norm, off 1
        proj = (dz * z).sum(1) / n
        shift = dz.sum(1) / n if layer else torch.zeros_like(proj)
        if layer:
            res["dbias"] = torch.ones_like(dy[:, 0]) @ dy
        res["dx"] = (dz - shift[:, None] - z * proj[:, None]) / sigma[:, None]
        res["dweight"] = torch.einsum("rc,rc->c", dy, z)
    return res


def _exact_embedding(s):
    ids = s["ids"].long()
    if not s["train"]:
        return s["weight"].double()[ids] * s["scale"]
    grad = torch.zeros(s["dtable"].shape, dtype=torch.float64, device=ids.device)
    live = torch.nonzero(ids != s["padding"])[:, 0]
    grad.index_put_((ids[live],), s["dy"].double()[live] * s["scale"], accumulate=True)
    return grad


def _exact_head_loss(s):
    labels = s["labels"].long()
    n, (v, c) = labels.numel(), s["weight"].shape
    if 6 * n * c * v > 14e12:  # over about 20 seconds of 64-bit products
        return None
    w = s["weight"].double()
    dev = w.device
    loss = torch.zeros(n, dtype=torch.float64, device=dev)
    lse = torch.zeros(n, dtype=torch.float64, device=dev)
    dh = torch.zeros(n, c, dtype=torch.float64, device=dev)
    dw = torch.zeros(v, c, dtype=torch.float64, device=dev)
    live = torch.nonzero(labels != IGNORE)[:, 0]
    for rows in live.split(2048):
        h = s["hidden"][rows].double()
        z = torch.einsum("td,vd->tv", h, w)
        lse[rows] = torch.logsumexp(z, 1)
        loss[rows] = lse[rows] - z[torch.arange(len(rows), device=dev), labels[rows]]
        if s["train"]:
            grad = torch.softmax(z, 1)
            grad[torch.arange(len(rows), device=dev), labels[rows]] -= 1
            grad *= s["dloss"][rows].double()[:, None]
            dh[rows] = torch.einsum("tv,vd->td", grad, w)
            dw += torch.einsum("tv,td->vd", grad, h)
    res = {"loss": loss, "lse": lse}
    if s["train"]:
        res.update(dhidden=dh, dweight=dw)
    return res


_EXACT = {"norm": _exact_norm, "embedding": _exact_embedding, "head_loss": _exact_head_loss}
