"""mfsdp_embedding_forward / _backward against the float64 oracle.

Forward is one product and one rounding: equal to the oracle's float64 product rounded to fp32
(and then to bf16).  Backward, with u = 2^-24: an id of k tokens is a sum of k terms, then one
product, so |d - ref| <= (k + 2) u scale sum |dy| elementwise, plus the rounding of a bf16
gradient (8 significant bits: 2^-8 of it).
"""

import numpy as np
import pytest
import torch

from oracle import embedding as oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


def _mat(rows, cols, dtype, gen, pitch=0, offset=0):
    base = torch.randn(rows * (cols + pitch) + offset, generator=gen, device="cuda")
    return base.to(TYPES[dtype])[offset:].view(rows, cols + pitch)[:, :cols]


def _ids(n, vocab, gen, how, index=torch.int64):
    if how == "uniform":
        ids = torch.randint(vocab, (n,), generator=gen, device="cuda")
    elif how == "one":
        ids = torch.full((n,), vocab - 1, device="cuda")
    elif how == "skew":    # half the tokens share one id, the rest fall off
        ids = (torch.rand(n, generator=gen, device="cuda") ** 6 * vocab).long().clamp_(max=vocab - 1)
        ids[torch.rand(n, generator=gen, device="cuda") < 0.5] = vocab // 2
    else:                  # every id in descending order
        ids = vocab - 1 - torch.arange(n, device="cuda") % vocab
    return ids.to(index)


@pytest.mark.parametrize("dim", [1, 8, 64, 100, 768, 1032])
@pytest.mark.parametrize("table,out", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"),
                                       ("bf16", "f32")])
def test_forward(dim, table, out):
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(dim)
    w = _mat(97, dim, table, gen)
    for n, index, scale in ((1, torch.int64, 1.0), (301, torch.int32, 11.3125)):
        ids = _ids(n, 97, gen, "uniform", index)
        o = torch.full((n, dim), float("nan"), dtype=TYPES[out], device="cuda")
        mfsdp.mfsdp_embedding_forward(w, ids, scale, o)
        ref = torch.from_numpy(oracle.forward(_np(w), ids.tolist(), scale)).float()
        assert torch.equal(o.cpu(), ref.to(TYPES[out]))


@pytest.mark.parametrize("pitch,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_forward_strides(pitch, offset):
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = _mat(50, 72, "bf16", gen, pitch, offset)
    ids = _ids(40, 50, gen, "uniform")
    o = _mat(40, 72, "bf16", gen, pitch, offset)
    mfsdp.mfsdp_embedding_forward(w, ids, 1.0, o)
    assert torch.equal(o, w[ids])


def test_forward_bad_ids():
    from matrix_optimizer_owner_gb300 import _lib, mfsdp
    w = torch.ones(10, 16, device="cuda")
    ids = torch.tensor([3, -1, 10, 9, 1 << 40], device="cuda")
    o = torch.empty(5, 16, device="cuda")
    mfsdp.mfsdp_embedding_forward(w, ids, 2.0, o)
    assert o[:, 0].tolist() == [2.0, 0.0, 0.0, 2.0, 0.0] and torch.equal(o, o[:, :1].expand(5, 16))
    assert _lib.STATUS_NAMES[mfsdp.mfsdp_query_status()] == "MFSDP_EINDEX"
    assert mfsdp.mfsdp_query_status() == 0


def _check(n, dim, vocab, how="uniform", dy="f32", grad="f32", scale=1.0, padding=-1,
           index=torch.int64, accumulate=False, seed=0, pitch=0, offset=0):
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = _ids(n, vocab, gen, how, index)
    d = _mat(n, dim, dy, gen, pitch, offset)
    g = _mat(vocab, dim, grad, gen, pitch, offset)
    if not accumulate:
        g.fill_(float("nan"))
    start = g.clone()
    mfsdp.mfsdp_embedding_backward(ids, d, scale, g, padding_idx=padding, accumulate=accumulate)
    ids_h, D = ids.tolist(), _np(d)
    s0 = _np(start) if accumulate else None
    ref = oracle.backward(ids_h, D, scale, vocab, padding, s0)
    mag = oracle.backward(ids_h, np.abs(D), scale, vocab, padding, np.abs(s0) if accumulate else None)
    count = np.bincount(ids_h, minlength=vocab)[:, None] if n else np.zeros((vocab, 1))
    tol = (count + 2) * U * mag
    if grad == "bf16":
        tol = tol + np.abs(ref) * 2.0 ** -8
    assert (np.abs(_np(g) - ref) <= tol).all()
    absent = count[:, 0] == 0
    if 0 <= padding < vocab:
        absent[padding] = True
    want = start if accumulate else torch.zeros_like(start)
    rows = torch.from_numpy(absent).cuda()
    assert torch.equal(g[rows], want[rows])          # untouched, or exactly zero
    again = start.clone() if accumulate else torch.empty_like(g)
    mfsdp.mfsdp_embedding_backward(ids, d, scale, again, padding_idx=padding, accumulate=accumulate)
    assert torch.equal(again, g)                     # repeats bit for bit
    assert mfsdp.mfsdp_query_status() == 0


# chunk boundaries (32 positions), one token, an empty call, more than one cluster step
@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 64, 65, 257, 3000])
@pytest.mark.parametrize("how", ["uniform", "one", "skew", "down"])
def test_backward_lengths(n, how):
    _check(n, 40, 61, how, seed=n)


@pytest.mark.parametrize("dim", [1, 7, 8, 64, 100, 768, 1024, 1032, 3000])
@pytest.mark.parametrize("dy,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_backward_widths_and_types(dim, dy, grad):
    _check(150, dim, 70, "skew", dy, grad, scale=3.5, seed=dim, index=torch.int32)


# places counted (up to 4096 tokens) and sorted, around the counting blocks' 64 tokens
@pytest.mark.parametrize("n", [2, 63, 64, 127, 1000, 4032, 4095, 4096, 4097, 9000])
@pytest.mark.parametrize("how", ["uniform", "skew", "down"])
def test_backward_counted_and_sorted(n, how):
    _check(n, 24, 700, how, seed=n, index=torch.int32 if n % 2 else torch.int64)
    _check(n, 24, 700, how, seed=n, padding=3, accumulate=True)


# a table whose zeros do not fit beside the sort: few tokens are sorted there too
@pytest.mark.parametrize("n", [1, 2000])
def test_backward_few_tokens_of_a_large_table(n):
    _check(n, 512, 90001, "skew", dy="bf16", grad="bf16", seed=n)


# one, two and three passes of the sort, at the digit boundaries, counted and sorted
@pytest.mark.parametrize("vocab", [1, 2, 511, 512, 513, 50257, 262143, 262144, 300001])
def test_backward_vocabularies_sorted(vocab):
    _check(4500, 16, vocab, "skew", seed=vocab)
    _check(4500, 16, vocab, "down", seed=vocab + 1)


@pytest.mark.parametrize("n", [300, 5000])
def test_backward_ids_outside_counted_and_sorted(n):
    from matrix_optimizer_owner_gb300 import _lib, mfsdp
    gen = torch.Generator(device="cuda").manual_seed(n)
    ids = _ids(n, 60, gen, "uniform")
    dy = _mat(n, 40, "f32", gen)
    keep = torch.rand(n, generator=gen, device="cuda") < 0.8
    want, got = (torch.empty(60, 40, device="cuda") for _ in range(2))
    zeroed = dy * keep[:, None]
    mfsdp.mfsdp_embedding_backward(ids, zeroed, 1.0, want)
    assert mfsdp.mfsdp_query_status() == 0
    bad = torch.tensor([60, -1, 1 << 40, -(1 << 40)], device="cuda")[torch.arange(n) % 4]
    dy[~keep] = float("nan")                         # not read into any row
    ids = torch.where(keep, ids, bad)
    mfsdp.mfsdp_embedding_backward(ids, dy, 1.0, got)
    assert _lib.STATUS_NAMES[mfsdp.mfsdp_query_status()] == "MFSDP_EINDEX"
    assert torch.allclose(got, want, rtol=0, atol=n * 2.0 ** -20)
    mfsdp.mfsdp_embedding_backward(torch.where(keep, ids, 60), dy, 1.0, got, padding_idx=60)
    assert mfsdp.mfsdp_query_status() == 0           # a padding id outside the table


# one, two and three passes of the sort, at the digit boundaries
@pytest.mark.parametrize("vocab", [1, 2, 511, 512, 513, 50257, 262143, 262144, 300001])
def test_backward_vocabularies(vocab):
    _check(500, 16, vocab, "skew", seed=vocab)
    _check(100, 16, vocab, "down", seed=vocab + 1)


def test_backward_padding_and_accumulate():
    _check(400, 48, 30, "skew", padding=15, seed=1)      # the id of half the tokens
    _check(400, 48, 30, "one", padding=29, seed=2)       # every token is padding
    _check(400, 48, 30, "uniform", accumulate=True, seed=3)
    _check(400, 48, 30, "skew", dy="bf16", grad="bf16", padding=0, accumulate=True, seed=4)
    _check(0, 48, 30, "uniform", accumulate=True, seed=5)


@pytest.mark.parametrize("pitch,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_backward_strides(pitch, offset):
    _check(200, 72, 90, "skew", dy="bf16", grad="f32", seed=6, pitch=pitch, offset=offset)


def test_backward_long_runs():
    # runs of thousands of tokens over many chunks; more tokens than the sort's threads
    _check(20000, 24, 7, "skew", seed=7)


def test_backward_bad_ids_take_no_part():
    from matrix_optimizer_owner_gb300 import _lib, mfsdp
    ids = torch.tensor([3, -1, 10, 3, 1 << 33, 9], device="cuda")
    d = torch.ones(6, 16, device="cuda")
    g = torch.empty(10, 16, device="cuda")
    mfsdp.mfsdp_embedding_backward(ids, d, 1.0, g)
    assert g[:, 0].tolist() == [0, 0, 0, 2, 0, 0, 0, 0, 0, 1]
    assert _lib.STATUS_NAMES[mfsdp.mfsdp_query_status()] == "MFSDP_EINDEX"
    # a padding id outside the table is not an error of its own
    mfsdp.mfsdp_embedding_backward(torch.tensor([3, -1], device="cuda"), d[:2], 1.0, g,
                                   padding_idx=-1)
    assert mfsdp.mfsdp_query_status() == 0 and g.sum().item() == 16


def test_backward_nan_stays_in_its_row():
    from matrix_optimizer_owner_gb300 import mfsdp
    ids = torch.tensor([1, 2, 3, 2], device="cuda")
    d = torch.ones(4, 16, device="cuda")
    d[1, 0] = float("nan")
    g = torch.empty(5, 16, device="cuda")
    mfsdp.mfsdp_embedding_backward(ids, d, 1.0, g)
    assert g.isnan().sum() == 1 and g[2, 0].isnan()
    mfsdp.mfsdp_embedding_backward(ids, d, 1.0, g, padding_idx=2)
    assert not g.isnan().any()                       # masked tokens leave nothing behind


def test_gradient_against_differences():
    """The lookup is linear in the table: <dE, V> = <lookup(V), dy> up to rounding."""
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(8)
    ids = _ids(120, 33, gen, "skew")
    d, v = _mat(120, 56, "f32", gen), _mat(33, 56, "f32", gen)
    g, o = torch.empty(33, 56, device="cuda"), torch.empty(120, 56, device="cuda")
    mfsdp.mfsdp_embedding_backward(ids, d, 0.75, g)
    mfsdp.mfsdp_embedding_forward(v, ids, 0.75, o)
    lhs, rhs = (g.double() * v.double()).sum().item(), (o.double() * d.double()).sum().item()
    mag = (o.double().abs() * d.double().abs()).sum().item()
    assert abs(lhs - rhs) <= 130 * U * mag


def test_other_stream_and_graph():
    from matrix_optimizer_owner_gb300 import mfsdp
    gen = torch.Generator(device="cuda").manual_seed(9)
    ids, d = _ids(300, 50, gen, "skew"), _mat(300, 64, "bf16", gen)
    g = torch.empty(50, 64, dtype=torch.bfloat16, device="cuda")
    mfsdp.mfsdp_embedding_backward(ids, d, 1.0, g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g2 = torch.empty_like(g)
    mfsdp.mfsdp_embedding_backward(ids, d, 1.0, g2, stream=s)
    s.synchronize()
    assert torch.equal(g2, g)
    g2.zero_()
    ws = torch.empty(mfsdp.mfsdp_embedding_backward_workspace_bytes(50, 64, 300),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mfsdp.mfsdp_embedding_backward(ids, d, 1.0, g2, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g2, g)


# the same, sorted by one block (up to 1024 tokens) and by the cluster
@pytest.mark.parametrize("n", [1, 31, 33, 500, 1023, 1024, 1025])
@pytest.mark.parametrize("how", ["uniform", "one", "down"])
def test_backward_few_tokens_of_a_large_table_sorted_by_one_block(n, how):
    _check(n, 264, 170001, how, dy="bf16", grad="bf16", seed=n, padding=5,
           index=torch.int32 if n % 2 else torch.int64)


@pytest.mark.parametrize("dim", [16, 17])                # rows of vectors, and others
@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -3.0])
def test_forward_bad_ids_give_zeros_at_any_scale(dim, scale):
    from matrix_optimizer_owner_gb300 import _lib, mfsdp
    w = torch.ones(10, dim, device="cuda")
    ids = torch.tensor([3, -1, 10], device="cuda")
    o = torch.empty(3, dim, device="cuda")
    mfsdp.mfsdp_embedding_forward(w, ids, scale, o)
    assert not o[1:].any() and not torch.signbit(o[1:]).any()
    assert torch.equal(o[:1], torch.full_like(o[:1], scale)) or o[:1].isnan().all()
    assert _lib.STATUS_NAMES[mfsdp.mfsdp_query_status()] == "MFSDP_EINDEX"
