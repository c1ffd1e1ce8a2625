"""The operators around a linear layer trained in 8 bits, as measured cases.

The owner step (``matrix_optimizer_owner_gb300.owner_step``) consumes the gradients of matrices.
The operators here are what a block computes to produce them, with the operands of its products
held in 8-bit floating point, one power-of-two scale for each group of 128 values:

``norm``        residual addition and layer or RMS norm, with the normalised rows in 8 bits (the
                next product's operand), and the backward pass, from the sum or from its 8-bit
                checkpoint;
``quantize``    8-bit matrices from 16- or 32-bit ones, in the groupings that the products take,
                and from an 8-bit checkpoint of another grouping;
``gemm``        products of 8-bit matrices: a layer's output, its input's gradient and its
                weight's gradient;
``activation``  SwiGLU and GELU with the result in 8 bits, and their backward pass from 8-bit
                checkpoints of the inputs, in both groupings that the products take.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once
at the end) or, where ``own`` is true, through the public entry points of the library.  An 8-bit
matrix is returned as its float8 values and its scales.
"""

from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-5
GROUP = 128
ROW, COL, TILE = 0, 1, 2        # scales of 1 x 128, 128 x 1 and 128 x 128 values
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
          "e5m2": torch.float8_e5m2}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}
TOP = {"e4m3": 8, "e5m2": 15}   # the largest value is 1.75 * 2^TOP


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One token through one norm of a Llama-3-8B block: a decoding step's smallest call, where
        # only latency counts.
        dict(name="norm_one_row_4096", op="norm", kind="rms", train=False, rows=1, cols=4096,
             dtype="bf16", params="bf16", fp8="e4m3", saved="h"),
        # A GPT-2-small training step's norm, 16 sequences of 1024 tokens, the block's input kept
        # for the backward pass in 8 bits.
        dict(name="norm_train_768", op="norm", kind="layer", train=True, rows=16384, cols=768,
             dtype="bf16", params="f32", fp8="e4m3", saved="h8"),
        # A Llama-3-8B training step's norm, the sum kept as it is.
        dict(name="norm_train_rms_4096", op="norm", kind="rms", train=True, rows=8192, cols=4096,
             dtype="bf16", params="bf16", fp8="e4m3", saved="h"),
        # The gradient of a Llama-3-8B gate layer's output, for both products of its backward pass.
        dict(name="quantize_grad_14336", op="quantize", source="bf16", rows=8192, cols=14336,
             fp8="e5m2", groups="row+col"),
        # The owner's fp32 master weight of a Llama-3-8B query projection, for all its products.
        dict(name="quantize_weight_4096", op="quantize", source="f32", rows=4096, cols=4096,
             fp8="e4m3", groups="tile"),
        # A norm's 8-bit output of an odd number of tokens, kept as a checkpoint, regrouped for the
        # weight's gradient.
        dict(name="regroup_checkpoint_odd", op="quantize", source="e4m3", rows=4099, cols=2000,
             fp8="e4m3", groups="col"),
        # One token through a Llama-3-8B gate layer: one pass over the weight.
        dict(name="gemm_one_token_14336", op="gemm", train=False, tokens=1, ins=4096, outs=14336,
             fp8="e4m3", grad="e4m3", dtype="bf16", wgrad="f32"),
        # The same layer's output for a training step.
        dict(name="gemm_forward_14336", op="gemm", train=False, tokens=8192, ins=4096, outs=14336,
             fp8="e4m3", grad="e4m3", dtype="bf16", wgrad="f32"),
        # The three products of a GPT-2-small qkv layer's training step.
        dict(name="gemm_train_768", op="gemm", train=True, tokens=16384, ins=768, outs=2304,
             fp8="e4m3", grad="e5m2", dtype="bf16", wgrad="f32"),
        # A few hundred tokens through a layer of odd sizes.
        dict(name="gemm_train_odd", op="gemm", train=True, tokens=333, ins=1001, outs=1500,
             fp8="e4m3", grad="e4m3", dtype="f32", wgrad="bf16"),
        # A Llama-3-8B MLP's SwiGLU in a training step.
        dict(name="activation_train_14336", op="activation", kind="swiglu", train=True, rows=8192,
             cols=14336, dtype="bf16", fp8="e4m3", grad="e5m2", saved="x8"),
        # A small odd GELU in fp32, its inputs kept as they are.
        dict(name="activation_train_f32_odd", op="activation", kind="gelu", train=True, rows=1001,
             cols=2005, dtype="f32", fp8="e4m3", grad="e4m3", saved="x"),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range: as often a multiple of 64 as not."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 64:
        n -= n % 64
    return max(lo, min(hi, n))


def draw(rng: random.Random):
    op = rng.choice(["norm", "quantize", "gemm", "gemm", "activation"])
    fp8, grad = rng.choice(["e4m3", "e4m3", "e5m2"]), rng.choice(["e4m3", "e5m2"])
    dtype, train = rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.7
    if op == "norm":
        return dict(op=op, kind=rng.choice(["layer", "rms"]), train=train,
                    rows=_size(rng, 1, 16384), cols=_size(rng, 64, 8192), dtype=dtype,
                    params=rng.choice(["f32", "bf16"]), fp8=fp8, saved=rng.choice(["h", "h8"]))
    if op == "quantize":
        source = rng.choice(["bf16", "f32", "e4m3"])
        return dict(op=op, source=source, rows=_size(rng, 1, 8192), cols=_size(rng, 64, 14336),
                    fp8="e4m3" if source == "e4m3" else fp8,
                    groups=rng.choice(["col", "tile"] if source == "e4m3" else
                                      ["row", "col", "tile", "row+col"]))
    if op == "activation":
        return dict(op=op, kind=rng.choice(["swiglu", "gelu"]), train=train,
                    rows=_size(rng, 1, 8192), cols=_size(rng, 64, 14336), dtype=dtype, fp8=fp8,
                    grad=grad, saved=rng.choice(["x", "x8"]))
    tokens, ins, outs = _size(rng, 1, 16384), _size(rng, 64, 8192), _size(rng, 64, 14336)
    most = 8192 * 4096 * 14336 // (3 if train else 1)
    tokens = min(tokens, max(1, most // (ins * outs)))
    return dict(op=op, train=train, tokens=tokens, ins=ins, outs=outs, fp8=fp8, grad=grad,
                dtype=dtype, wgrad=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------------------------------ 8 bits
def _blocks(n):
    return -(-n // GROUP)


def _spread(scales, groups, rows, cols):
    """A value per element from one per group."""
    if groups in (COL, TILE):
        scales = scales.repeat_interleave(GROUP, 0)[:rows]
    if groups in (ROW, TILE):
        scales = scales.repeat_interleave(GROUP, 1)[:, :cols]
    return scales


def _pitched(rows, cols, dtype):
    """A byte matrix whose rows start on 16-byte boundaries."""
    return torch.empty(rows, -(-cols // 16) * 16, dtype=dtype, device="cuda")[:, :cols]


def _scale_shape(groups, rows, cols):
    return (_blocks(rows) if groups in (COL, TILE) else rows,
            _blocks(cols) if groups in (ROW, TILE) else cols)


def _empty8(rows, cols, groups, fp8):
    return (_pitched(rows, cols, DTYPES[fp8]),
            torch.empty(_scale_shape(groups, rows, cols), dtype=torch.float8_e8m0fnu,
                        device="cuda"))


def _quantized(v, groups, fp8):
    """fp32 values as float8 ones and their groups' scales: the least powers of two (from 2^-127)
    that bring a group's largest value within the type's range."""
    rows, cols = v.shape
    gr, gc = _scale_shape(groups, rows, cols)
    pr = gr * GROUP if groups in (COL, TILE) else rows
    pc = gc * GROUP if groups in (ROW, TILE) else cols
    a = torch.nn.functional.pad(v.abs(), (0, pc - cols, 0, pr - rows))
    top = a.view(gr, pr // gr, gc, pc // gc).amax((1, 3))
    frac, e = torch.frexp(top)
    e = e - 1 - TOP[fp8] + (frac > 0.875)
    e = torch.where(top > 0, e, -127).clamp_(min=-127)
    q = torch.ldexp(v, -_spread(e, groups, rows, cols)).to(DTYPES[fp8])
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(q, s, groups):
    return q.float() * _spread(s.float(), groups, *q.shape)


def _held(v, groups, fp8):
    """An input that is held in 8 bits, in a buffer as the framework lays them out."""
    q, s = _quantized(v, groups, fp8)
    data = _pitched(*v.shape, q.dtype)
    data.copy_(q)
    return data, s


# ------------------------------------------------------------------------------------ inputs
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
        layer = case["kind"] == "layer"
        # a residual stream: rows of different scale, off centre, and a branch added to it
        stream = normal(r, c) * normal(r, 1, std=0.5).exp() + normal(r, 1, std=0.3)
        s.update(x=normal(r, c, std=0.5, dtype=d), residual=stream.to(DTYPES[d]),
                 weight=normal(c, std=0.1, mean=1.0, dtype=p),
                 bias=normal(c, std=0.1, dtype=p) if layer else None, h=out(r, c, dtype=d),
                 y8=_empty8(r, c, ROW, case["fp8"]), mean=out(r) if layer else None, rstd=out(r),
                 h8=_empty8(r, c, ROW, case["fp8"]) if case["saved"] == "h8" else None)
        if case["train"]:
            s.update(dy=normal(r, c, std=1e-3, dtype=d), dres=normal(r, c, std=1e-3, dtype=d),
                     dx=out(r, c, dtype=d), dweight=out(c, dtype=p),
                     dbias=out(c, dtype=p) if layer else None)
        return s
    if case["op"] == "quantize":
        r, c, src = case["rows"], case["cols"], case["source"]
        # values as a layer has them: tokens and features of different scale
        v = normal(r, c) * normal(r, 1, std=0.7).exp() * normal(1, c, std=0.7).exp()
        s.update(x=_held(v, ROW, src) if src in TOP else v.to(DTYPES[src]),
                 out=[_empty8(r, c, g, case["fp8"]) for g in _groups(case)])
        return s
    if case["op"] == "activation":
        r, c, d = case["rows"], case["cols"], case["dtype"]
        x8 = case["saved"] == "x8"
        pair = case["kind"] == "swiglu"
        s.update(gate=normal(r, c, dtype=d), up=normal(r, c, dtype=d) if pair else None,
                 y8=_empty8(r, c, ROW, case["fp8"]),
                 gate8=_empty8(r, c, ROW, case["fp8"]) if x8 else None,
                 up8=_empty8(r, c, ROW, case["fp8"]) if x8 and pair else None)
        if case["train"]:
            s.update(dy=normal(r, c, std=1e-3, dtype=d),
                     grads=[[_empty8(r, c, g, case["grad"]) for g in (ROW, COL)]
                            for _ in range(2 if pair else 1)])
        return s
    t, k, n = case["tokens"], case["ins"], case["outs"]
    # normalised activations with outlying features, against a weight that keeps their scale
    x = normal(t, k) * normal(1, k, std=0.5).exp()
    w = normal(n, k, std=1.0 / math.sqrt(k))
    s.update(x=_held(x, ROW, case["fp8"]), w=_held(w, TILE, case["fp8"]),
             y=out(t, n, dtype=case["dtype"]))
    if case["train"]:
        dy = normal(t, n, std=1e-3) * normal(t, 1, std=0.5).exp()
        s.update(x_col=_held(x, COL, case["fp8"]), dy=_held(dy, ROW, case["grad"]),
                 dy_col=_held(dy, COL, case["grad"]), dx=out(t, k, dtype=case["dtype"]),
                 dw=out(n, k, dtype=case["wgrad"]))
    return s


def _groups(case):
    return [{"row": ROW, "col": COL, "tile": TILE}[g] for g in case["groups"].split("+")]


# ------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _RUN_OWN[state["op"]](state)
    with torch.no_grad():
        return _RUN_PLAIN[state["op"]](state)


def _plain_norm(s):
    layer, d = s["kind"] == "layer", s["x"].dtype
    h = s["x"].float() + s["residual"].float()
    mean = h.mean(1) if layer else None
    hc = h - mean[:, None] if layer else h
    rstd = ((hc * hc).mean(1) + EPS).rsqrt()
    w = s["weight"].float()
    y = hc * rstd[:, None] * w
    if layer:
        y = y + s["bias"].float()
    res = {"h": h.to(d), "y8": _quantized(y, ROW, s["fp8"]), "rstd": rstd}
    if layer:
        res["mean"] = mean
    if s["saved"] == "h8":
        res["h8"] = _quantized(h, ROW, s["fp8"])
    if s["train"]:
        kept = _values(*res["h8"], ROW) if s["saved"] == "h8" else res["h"].float()
        z = (kept - mean[:, None] if layer else kept) * rstd[:, None]
        dy = s["dy"].float()
        g = dy * w
        dx = g - z * (g * z).mean(1, keepdim=True)
        if layer:
            dx = dx - g.mean(1, keepdim=True)
            res["dbias"] = dy.sum(0).to(s["weight"].dtype)
        res["dx"] = (dx * rstd[:, None] + s["dres"].float()).to(d)
        res["dweight"] = (dy * z).sum(0).to(s["weight"].dtype)
    return res


def _plain_quantize(s):
    v = _values(*s["x"], ROW) if s["source"] in TOP else s["x"].float()
    return [_quantized(v, g, s["fp8"]) for g in _groups(s)]


def _plain_gemm(s):
    x, w = _values(*s["x"], ROW), _values(*s["w"], TILE)
    res = {"y": (x @ w.T).to(s["y"].dtype)}
    if s["train"]:
        res["dx"] = (_values(*s["dy"], ROW) @ w).to(s["dx"].dtype)
        res["dw"] = (_values(*s["dy_col"], COL).T @ _values(*s["x_col"], COL)).to(s["dw"].dtype)
    return res


def _plain_activation(s):
    gate, up = s["gate"].float(), None if s["up"] is None else s["up"].float()
    res = {}
    if s["kind"] == "swiglu":
        y = gate / (1 + (-gate).exp()) * up
    else:
        y = 0.5 * gate * (1 + torch.tanh(0.7978845608028654 * (gate + 0.044715 * gate ** 3)))
    res["y8"] = _quantized(y, ROW, s["fp8"])
    if s["saved"] == "x8":
        res["gate8"] = _quantized(gate, ROW, s["fp8"])
        gate = _values(*res["gate8"], ROW)
        if up is not None:
            res["up8"] = _quantized(up, ROW, s["fp8"])
            up = _values(*res["up8"], ROW)
    if s["train"]:
        dy = s["dy"].float()
        if s["kind"] == "swiglu":
            p = 1 / (1 + (-gate).exp())
            grads = [dy * up * p * (1 + gate * (1 - p)), dy * gate * p]
        else:
            t = torch.tanh(0.7978845608028654 * (gate + 0.044715 * gate ** 3))
            inner = 0.7978845608028654 * (1 + 3 * 0.044715 * gate ** 2)
            grads = [dy * (0.5 * (1 + t) + 0.5 * gate * (1 - t * t) * inner)]
        res["grads"] = [[_quantized(g, k, s["grad"]) for k in (ROW, COL)] for g in grads]
    return res


def _own_matrix(mfsdp, held, groups):
    return None if held is None else mfsdp.Fp8Matrix(held[0], held[1], groups)


def _own_norm(s):
    from matrix_optimizer_owner_gb300 import mfsdp
    layer = s["kind"] == "layer"
    kind = mfsdp.NORM_LAYER if layer else mfsdp.NORM_RMS
    h8 = _own_matrix(mfsdp, s["h8"], ROW)
    mfsdp.mfsdp_norm_residual_forward(kind, s["x"], s["residual"], s["weight"], s["bias"], EPS,
                                      h=s["h"], y8=_own_matrix(mfsdp, s["y8"], ROW), h8=h8,
                                      mean=s["mean"], rstd=s["rstd"])
    names = ["h", "y8", "rstd"] + (["mean"] if layer else []) + (["h8"] if h8 else [])
    if s["train"]:
        mfsdp.mfsdp_norm_residual_backward(kind, s["dy"], s["dres"], h8 or s["h"], s["weight"],
                                           s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"])
        names += ["dx", "dweight"] + (["dbias"] if layer else [])
    return {k: s[k] for k in names}


def _own_quantize(s):
    from matrix_optimizer_owner_gb300 import mfsdp
    out = [_own_matrix(mfsdp, o, g) for o, g in zip(s["out"], _groups(s))]
    if s["source"] in TOP:
        mfsdp.mfsdp_regroup_fp8(_own_matrix(mfsdp, s["x"], ROW), *out)
    else:
        mfsdp.mfsdp_quantize_fp8(s["x"], *out)
    return s["out"]


def _own_gemm(s):
    from matrix_optimizer_owner_gb300 import mfsdp
    x, w = _own_matrix(mfsdp, s["x"], ROW), _own_matrix(mfsdp, s["w"], TILE)
    mfsdp.mfsdp_gemm_fp8(x, w, s["y"], trans_b=True)
    if not s["train"]:
        return {"y": s["y"]}
    mfsdp.mfsdp_gemm_fp8(_own_matrix(mfsdp, s["dy"], ROW), w, s["dx"])
    mfsdp.mfsdp_gemm_fp8(_own_matrix(mfsdp, s["dy_col"], COL),
                         _own_matrix(mfsdp, s["x_col"], COL), s["dw"], trans_a=True)
    return {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}


def _own_activation(s):
    from matrix_optimizer_owner_gb300 import mfsdp
    kind = mfsdp.ACT_SWIGLU if s["kind"] == "swiglu" else mfsdp.ACT_GELU
    gate8, up8 = (_own_matrix(mfsdp, s[k], ROW) for k in ("gate8", "up8"))
    mfsdp.mfsdp_activation_forward(kind, s["gate"], s["up"], y8=_own_matrix(mfsdp, s["y8"], ROW),
                                   gate8=gate8, up8=up8)
    names = ["y8"] + (["gate8"] if gate8 else []) + (["up8"] if up8 else [])
    if s["train"]:
        g = [[_own_matrix(mfsdp, m, k) for m, k in zip(both, (ROW, COL))] for both in s["grads"]]
        g += [[None, None]] * (2 - len(g))
        mfsdp.mfsdp_activation_backward(kind, s["dy"], gate8 or s["gate"], up8 or s["up"],
                                        dgate8=g[0][0], dgate8_col=g[0][1], dup8=g[1][0],
                                        dup8_col=g[1][1])
        names.append("grads")
    return {k: s[k] for k in names}


_RUN_PLAIN = {"norm": _plain_norm, "quantize": _plain_quantize, "gemm": _plain_gemm,
              "activation": _plain_activation}
_RUN_OWN = {"norm": _own_norm, "quantize": _own_quantize, "gemm": _own_gemm,
            "activation": _own_activation}


# ------------------------------------------------------------------------------------ work
def _bytes8(groups, rows, cols):
    gr, gc = _scale_shape(groups, rows, cols)
    return rows * cols + gr * gc


def work(case):
    if case["op"] == "gemm":
        t, k, n, c = case["tokens"], case["ins"], case["outs"], BYTES[case["dtype"]]
        total = _bytes8(ROW, t, k) + _bytes8(TILE, n, k) + t * n * c
        if not case["train"]:
            return {"bytes": total, "flops": 2 * t * k * n}
        total += (_bytes8(COL, t, k) + _bytes8(ROW, t, n) + _bytes8(COL, t, n) + t * k * c
                  + n * k * BYTES[case["wgrad"]])
        return {"bytes": total, "flops": 6 * t * k * n}
    r, c = case["rows"], case["cols"]
    n = r * c
    row8, col8 = _bytes8(ROW, r, c), _bytes8(COL, r, c)
    if case["op"] == "quantize":
        src = row8 if case["source"] in TOP else n * BYTES[case["source"]]
        return {"bytes": src + sum(_bytes8(g, r, c) for g in _groups(case)), "flops": 4 * n}
    e = n * BYTES[case["dtype"]]
    if case["op"] == "norm":
        layer, x8 = case["kind"] == "layer", case["saved"] == "h8"
        params = c * BYTES[case["params"]] * (2 if layer else 1)
        total = 3 * e + row8 * (2 if x8 else 1) + params + r * 4 * (2 if layer else 1)
        # backward: what was kept is an output of the pass already, so dy and dres in, dx out
        return {"bytes": total + (3 * e + params if case["train"] else 0),
                "flops": (24 if case["train"] else 10) * n}
    pair = 2 if case["kind"] == "swiglu" else 1
    total = pair * e + row8 * (1 + (pair if case["saved"] == "x8" else 0))
    return {"bytes": total + (e + pair * (row8 + col8) if case["train"] else 0),
            "flops": (40 if case["train"] else 15) * n}


# ------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """What ``run`` returns, from the definitions in 64 bits."""
    return _EXACT[case["op"]](prepare(case, seed))


def _exact_quantized(v, groups, fp8):
    rows, cols = v.shape
    mantissa, least = (3, -6) if fp8 == "e4m3" else (2, -14)
    biggest = 448.0 if fp8 == "e4m3" else 57344.0
    a = v.abs()
    if groups in (ROW, TILE):
        a = torch.stack([p.amax(1) for p in a.split(GROUP, 1)], 1)
    if groups in (COL, TILE):
        a = torch.stack([p.amax(0) for p in a.split(GROUP, 0)], 0)
    e = torch.full_like(a, -127.0)
    some = a > 0
    e[some] = torch.ceil(torch.log2(a[some] / biggest))
    # the logarithm's rounding at a border
    e = torch.where(a > biggest * torch.exp2(e), e + 1, e)
    e = torch.where(a <= biggest * torch.exp2(e - 1), e - 1, e).clamp(min=-127)
    u = v / torch.exp2(_spread(e, groups, rows, cols))
    # steps of 2^-mantissa of the value's power of two, and fixed ones below the least normal
    power = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** least)))
    step = torch.exp2(power - mantissa)
    return torch.round(u / step) * step, torch.exp2(e)


def _exact_values(held, groups):
    q, s = held
    v = q.double()
    rows, cols = v.shape
    i = torch.arange(rows, device=v.device)[:, None]
    j = torch.arange(cols, device=v.device)[None, :]
    return v * s.double()[i // GROUP if groups != ROW else i, j // GROUP if groups != COL else j]


def _exact_norm(s):
    layer = s["kind"] == "layer"
    h = s["x"].double() + s["residual"].double()
    n = h.shape[1]
    mu = h.sum(1) / n if layer else torch.zeros_like(h[:, 0])
    sigma = torch.sqrt(((h - mu[:, None]) ** 2).sum(1) / n + EPS)
    w = s["weight"].double()
    y = (h - mu[:, None]) / sigma[:, None] * w
    if layer:
        y = y + s["bias"].double()
    res = {"h": h, "y8": _exact_quantized(y, ROW, s["fp8"]), "rstd": 1 / sigma}
    if layer:
        res["mean"] = mu
    kept = h.to(s["x"].dtype).double()
    if s["saved"] == "h8":
        q, e = res["h8"] = _exact_quantized(h, ROW, s["fp8"])
        kept = q * _spread(e, ROW, *q.shape)
    if s["train"]:
        z = (kept - mu[:, None]) / sigma[:, None]
        dy = s["dy"].double()
        dz = dy * w
        # the projection off z and, for a layer norm, off 1, beside the residual's own gradient
        proj = (dz * z).sum(1) / n
        shift = dz.sum(1) / n if layer else torch.zeros_like(proj)
        if layer:
            res["dbias"] = torch.ones_like(dy[:, 0]) @ dy
        res["dx"] = s["dres"].double() + (dz - shift[:, None] - z * proj[:, None]) / sigma[:, None]
        res["dweight"] = torch.einsum("rc,rc->c", dy, z)
    return res


def _exact_quantize(s):
    v = _exact_values(s["x"], ROW) if s["source"] in TOP else s["x"].double()
    return [_exact_quantized(v, g, s["fp8"]) for g in _groups(s)]


def _exact_gemm(s):
    w = _exact_values(s["w"], TILE)
    res = {"y": torch.einsum("tk,nk->tn", _exact_values(s["x"], ROW), w)}
    if s["train"]:
        res["dx"] = torch.einsum("tn,nk->tk", _exact_values(s["dy"], ROW), w)
        res["dw"] = torch.einsum("tn,tk->nk", _exact_values(s["dy_col"], COL),
                                 _exact_values(s["x_col"], COL))
    return res


def _exact_activation(s):
    def act(g, u):
        if s["kind"] == "swiglu":
            return g * torch.sigmoid(g) * u
        return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))

    gate = s["gate"].double()
    up = None if s["up"] is None else s["up"].double()
    res = {"y8": _exact_quantized(act(gate, up), ROW, s["fp8"])}
    if s["saved"] == "x8":
        q, e = res["gate8"] = _exact_quantized(gate, ROW, s["fp8"])
        gate = q * _spread(e, ROW, *q.shape)
        if up is not None:
            q, e = res["up8"] = _exact_quantized(up, ROW, s["fp8"])
            up = q * _spread(e, ROW, *q.shape)
    if s["train"]:
        leaves = [t.requires_grad_() for t in (gate, up) if t is not None]
        with torch.enable_grad():
            grads = torch.autograd.grad(act(gate, up), leaves, s["dy"].double())
        res["grads"] = [[_exact_quantized(g, k, s["grad"]) for k in (ROW, COL)] for g in grads]
    return res


_EXACT = {"norm": _exact_norm, "quantize": _exact_quantize, "gemm": _exact_gemm,
          "activation": _exact_activation}
