"""Host-side checks of the norm, embedding and head-loss entry points: refusals before any launch, and
workspace sizes.  Pointers here are made-up addresses that no kernel ever sees."""

import ctypes as C
import os

import pytest

P = 4096          # an address with every alignment
EINVAL, ESHAPE, EALIGN, EWORKSPACE = -1, -2, -3, -5


@pytest.fixture(scope="module")
def lib():
    from matrix_optimizer_owner_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from matrix_optimizer_owner_gb300 import build
        build.build()
    return _lib.load()


def _call(fn, good, **changes):
    args = dict(good, **changes)
    assert set(args) == set(good)
    return fn(*args.values())


NORM_FWD = dict(kind=0, rows=4, cols=64, dtype=1, pdtype=0, x=P, ld_x=64, w=P, b=P, eps=1e-5, y=P,
                ld_y=64, mean=P, rstd=P, stream=None)
NORM_BWD = dict(kind=0, rows=4, cols=64, dtype=1, pdtype=0, dy=P, ld_dy=64, x=P, ld_x=64, w=P,
                mean=P, rstd=P, dx=P, ld_dx=64, dw=P, db=P, ws=P, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(kind=2), EINVAL), (dict(dtype=2), EINVAL), (dict(pdtype=-1), EINVAL),
    (dict(rows=-1), ESHAPE), (dict(cols=0), ESHAPE), (dict(cols=1 << 31), ESHAPE),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(x=None), EINVAL),
    (dict(y=None), EINVAL), (dict(ld_x=63), EINVAL), (dict(ld_y=63), EINVAL),
    (dict(kind=1, mean=None), EINVAL),            # an RMS norm with a bias
    (dict(kind=1, b=None), EINVAL),               # an RMS norm with a mean
    (dict(x=P + 1), EALIGN), (dict(w=P + 2), EALIGN), (dict(rstd=P + 2), EALIGN),
    (dict(rows=0, x=None, y=None), 0),
])
def test_norm_forward_refusals(lib, change, status):
    assert _call(lib.mfsdp_norm_forward, NORM_FWD, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(kind=-1), EINVAL), (dict(dtype=5), EINVAL), (dict(rows=1 << 31), ESHAPE),
    (dict(dy=None), EINVAL), (dict(x=None), EINVAL), (dict(dx=None), EINVAL),
    (dict(rstd=None), EINVAL), (dict(mean=None), EINVAL), (dict(ld_dx=10), EINVAL),
    (dict(kind=1, mean=None), EINVAL),            # an RMS norm with a bias gradient
    (dict(ws=None), EINVAL), (dict(ws=P + 8), EALIGN), (dict(dy=P + 1), EALIGN),
    (dict(ws_bytes=0), EWORKSPACE), (dict(ws_bytes=4 * 2 * 64 * 4 - 1), EWORKSPACE),
])
def test_norm_backward_refusals(lib, change, status):
    assert _call(lib.mfsdp_norm_backward, NORM_BWD, **change) == status


def test_norm_workspace(lib):
    from matrix_optimizer_owner_gb300 import mfsdp
    assert mfsdp.mfsdp_norm_backward_workspace_bytes(4, 64) == 4 * 2 * 64 * 4
    # bounded by the blocks of a launch, not by the rows
    assert (mfsdp.mfsdp_norm_backward_workspace_bytes(1 << 20, 64)
            == mfsdp.mfsdp_norm_backward_workspace_bytes(1 << 30, 64))
    out = C.c_size_t(0)
    assert lib.mfsdp_norm_backward_workspace_bytes(4, 0, C.byref(out)) == ESHAPE
    assert lib.mfsdp_norm_backward_workspace_bytes(4, 64, None) == EINVAL


EMB_FWD = dict(vocab=100, dim=64, tdtype=0, table=P, ld_t=64, n=5, idtype=1, ids=P, scale=1.0,
               odtype=1, out=P, ld_o=64, stream=None)
EMB_BWD = dict(vocab=100, dim=64, n=5, idtype=1, ids=P, pad=-1, scale=1.0, dydtype=1, dy=P,
               ld_dy=64, acc=0, gdtype=1, dt=P, ld_dt=64, ws=P, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(vocab=0), ESHAPE), (dict(dim=0), ESHAPE), (dict(n=-1), ESHAPE),
    (dict(vocab=1 << 31), ESHAPE), (dict(tdtype=2), EINVAL), (dict(odtype=2), EINVAL),
    (dict(idtype=2), EINVAL), (dict(table=None), EINVAL), (dict(ids=None), EINVAL),
    (dict(out=None), EINVAL), (dict(ld_t=63), EINVAL), (dict(ld_o=1), EINVAL),
    (dict(table=P + 2), EALIGN), (dict(ids=P + 4), EALIGN), (dict(out=P + 1), EALIGN),
    (dict(n=0, table=None, ids=None, out=None), 0),
])
def test_embedding_forward_refusals(lib, change, status):
    assert _call(lib.mfsdp_embedding_forward, EMB_FWD, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(vocab=0), ESHAPE), (dict(n=(1 << 31) - 1), ESHAPE), (dict(dydtype=2), EINVAL),
    (dict(gdtype=7), EINVAL), (dict(idtype=-1), EINVAL), (dict(dt=None), EINVAL),
    (dict(dy=None), EINVAL), (dict(ids=None), EINVAL), (dict(ld_dy=2), EINVAL),
    (dict(ld_dt=2), EINVAL), (dict(ws=None), EINVAL), (dict(ws=P + 16), EALIGN),
    (dict(dt=P + 1), EALIGN), (dict(ws_bytes=256), EWORKSPACE),
])
def test_embedding_backward_refusals(lib, change, status):
    assert _call(lib.mfsdp_embedding_backward, EMB_BWD, **change) == status


def test_embedding_workspace(lib):
    from matrix_optimizer_owner_gb300 import mfsdp
    need = mfsdp.mfsdp_embedding_backward_workspace_bytes(100, 64, 5)
    assert need % 256 == 0 and need >= 5 * 16 + 100 + 2 * 64 * 4
    assert _call(lib.mfsdp_embedding_backward, EMB_BWD, ws_bytes=need - 1) == EWORKSPACE
    out = C.c_size_t(0)
    assert lib.mfsdp_embedding_backward_workspace_bytes(0, 64, 5, C.byref(out)) == ESHAPE
    assert lib.mfsdp_embedding_backward_workspace_bytes(1, 64, 5, None) == EINVAL


HEAD_FWD = dict(n=5, dim=64, vocab=100, dtype=1, h=P, ld_h=64, w=P, ld_w=64, idtype=1, lab=P,
                ignore=-100, loss=P, lse=P, ws=P, ws_bytes=1 << 30, stream=None)
HEAD_BWD = dict(n=5, dim=64, vocab=100, dtype=1, h=P, ld_h=64, w=P, ld_w=64, idtype=1, lab=P,
                ignore=-100, lse=P, dl=P, piece=0, dh=P, ld_dh=64, dw=P, ld_dw=64, ws=P,
                ws_bytes=1 << 30, stream=None)
HEAD_BOTH = [
    (dict(n=-1), ESHAPE), (dict(dim=0), ESHAPE), (dict(vocab=0), ESHAPE),
    (dict(vocab=(1 << 30) + 1), ESHAPE), (dict(dtype=2), EINVAL), (dict(idtype=2), EINVAL),
    (dict(h=None), EINVAL), (dict(w=None), EINVAL), (dict(lab=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(ld_h=63), EINVAL), (dict(ld_w=63), EINVAL),
    (dict(h=P + 1), EALIGN), (dict(w=P + 1), EALIGN), (dict(lab=P + 4), EALIGN),
    (dict(lse=P + 2), EALIGN), (dict(ws=P + 64), EALIGN), (dict(ws_bytes=1024), EWORKSPACE),
]


@pytest.mark.parametrize("change,status", HEAD_BOTH + [
    (dict(loss=P + 1), EALIGN), (dict(n=0, h=None, lab=None, loss=None, lse=None), 0)])
def test_head_loss_forward_refusals(lib, change, status):
    assert _call(lib.mfsdp_head_loss_forward, HEAD_FWD, **change) == status


@pytest.mark.parametrize("change,status", HEAD_BOTH + [
    (dict(piece=-1), EINVAL), (dict(piece=1 << 31), ESHAPE), (dict(lse=None), EINVAL),
    (dict(dl=None), EINVAL), (dict(ld_dh=1), EINVAL), (dict(ld_dw=1), EINVAL),
    (dict(dh=P + 1), EALIGN), (dict(dw=P + 1), EALIGN), (dict(dl=P + 1), EALIGN),
    (dict(dh=None, dw=None), 0)])
def test_head_loss_backward_refusals(lib, change, status):
    assert _call(lib.mfsdp_head_loss_backward, HEAD_BWD, **change) == status


def test_head_loss_workspace(lib):
    def need(n, dim, vocab, dtype, backward, w=P, ld=None, piece=0):
        out = C.c_size_t(0)
        assert lib.mfsdp_head_loss_workspace_bytes(n, dim, vocab, dtype, backward, w, ld or dim,
                                                   piece, C.byref(out)) == 0
        return out.value
    # the logits of 8192 tokens over 128256 entries would take 2.1 GB in bf16; a piece of the
    # gradient, the compacted hidden rows and the fp32 sums of dhidden take a fraction
    assert need(8192, 4096, 128256, 1, 1) < 400 << 20
    assert need(8192, 4096, 128256, 1, 0) < 150 << 20
    assert need(8192, 4096, 128256, 1, 1, piece=1024) < need(8192, 4096, 128256, 1, 1)
    # an unaligned weight adds the copy of one piece
    assert need(64, 100, 5000, 1, 0, ld=101) > need(64, 100, 5000, 1, 0, ld=104)
    assert need(64, 100, 5000, 1, 0, w=P + 2, ld=104) > need(64, 100, 5000, 1, 0, ld=104)
    out = C.c_size_t(0)
    f = lib.mfsdp_head_loss_workspace_bytes
    assert f(5, 64, 100, 3, 0, P, 64, 0, C.byref(out)) == EINVAL
    assert f(5, 64, 100, 1, 0, P, 32, 0, C.byref(out)) == EINVAL
    assert f(5, 64, 0, 1, 0, P, 64, 0, C.byref(out)) == ESHAPE
    assert f(5, 64, 100, 1, 0, P, 64, 0, None) == EINVAL


def test_binding_refuses_wrong_tensors():
    import torch

    from matrix_optimizer_owner_gb300 import mfsdp
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA device"):      # host tensors
        mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x, w, None, 1e-5, x)
    with pytest.raises(TypeError):
        mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x.half(), w, None, 1e-5, x.half())
    with pytest.raises(TypeError):
        mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x, w, w.bfloat16(), 1e-5, x)
    with pytest.raises(ValueError):
        mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x, torch.zeros(9), None, 1e-5, x)
    with pytest.raises(ValueError):
        mfsdp.mfsdp_norm_forward(mfsdp.NORM_LAYER, x, w, None, 1e-5, torch.zeros(8, 4).T)
    table, ids = torch.zeros(10, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        mfsdp.mfsdp_embedding_forward(table, ids.short(), 1.0, x)
    with pytest.raises(ValueError):
        mfsdp.mfsdp_embedding_forward(table, ids[:3], 1.0, x)
    with pytest.raises(ValueError, match="CUDA device"):
        mfsdp.mfsdp_embedding_backward(ids, x, 1.0, table)
    lab, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(TypeError):                            # two dtypes
        mfsdp.mfsdp_head_loss_forward(x, table.bfloat16(), lab, f, f)
    with pytest.raises(ValueError):                           # widths differ
        mfsdp.mfsdp_head_loss_forward(x, torch.zeros(10, 9), lab, f, f)
    with pytest.raises(TypeError):                            # loss not fp32
        mfsdp.mfsdp_head_loss_forward(x, table, lab, f.double(), f)
    with pytest.raises(ValueError, match="CUDA device"):
        mfsdp.mfsdp_head_loss_backward(x, table, lab, f, f, x, table)


@pytest.mark.parametrize("as_handle", [False, True])
def test_fresh_workspace_comes_from_the_stream_it_is_used_on(monkeypatch, as_handle):
    import contextlib

    import torch

    from matrix_optimizer_owner_gb300 import mfsdp
    current, made_on = ["default"], []

    class Stream:
        cuda_stream = 77

    @contextlib.contextmanager
    def switch(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    class Like:
        def new_empty(self, shape, dtype):
            made_on.append(current[-1])
            return torch.empty(shape, dtype=torch.uint8)

    class External(Stream):
        def __init__(self, handle):
            assert handle == 77

    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(mfsdp, "_is_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    ws, size = mfsdp._workspace(None, 100, Like(), 0, 77 if as_handle else Stream(), 77)
    assert made_on == [77] and ws.numel() == size == 100
    # on the current stream: a large one is fresh and made there
    mfsdp._workspace(None, mfsdp._Scratch.LIMIT + 1, Like(), 0, None, 5)
    assert made_on == [77, "default"] and current == ["default"]


def test_gemm_workspace_comes_from_the_stream_it_is_used_on(monkeypatch):
    import contextlib

    import torch

    from matrix_optimizer_owner_gb300 import mfsdp
    current, made_on = ["default"], []

    class Stream:
        cuda_stream = 77

    class FakeLib:                       # no kernel sees these host tensors
        def mfsdp_gemm_f32_workspace_bytes(self, n):
            return 256 * n

        def mfsdp_gemm_f32_batched(self, *args):
            assert args[-1] == 77
            return 0

    @contextlib.contextmanager
    def switch(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def recorded(f):
        def g(*args, **kw):
            made_on.append(current[-1])
            return f(*args, **kw)
        return g

    a = torch.zeros(4, 4)
    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(mfsdp._lib, "load", FakeLib)
    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    monkeypatch.setattr(torch.Tensor, "new_empty", recorded(torch.Tensor.new_empty))
    mfsdp.mfsdp_gemm_f32_batched([(a, a, a.clone(), 1.0, 0.0)], stream=Stream())
    assert made_on == [77]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("n", [16, 64, 333, 1000, 4096, 32768])
@pytest.mark.parametrize("dim,ld", [(768, 768), (1024, 1024), (4096, 4096), (4096, 4099), (4090, 4090),
                                    (4095, 4095), (16384, 16384)])
@pytest.mark.parametrize("vocab", [50257, 128256])
def test_head_loss_workspace_is_bounded(lib, dtype, n, dim, ld, vocab):
    """Whatever the rows' alignment: the backward pass 400 MiB (an fp32 W's bytes, for one wave of
    columns at most, where that is more), or what does not depend on the piece with 128 MiB or 4096
    columns; forward a copy of hidden with 64 MiB (bf16) or 128 MiB (fp32), with a copied W 390 MiB or
    a wave of an fp32 W's rows, or with 4096 columns.  A piece is rounded up to a whole tile, 1/16 of
    the least one."""
    def need(backward, piece):
        out = C.c_size_t(0)
        assert lib.mfsdp_head_loss_workspace_bytes(n, dim, vocab, dtype, backward, P, ld, piece,
                                                   C.byref(out)) == 0
        return out.value

    rows, pitch, es = (n + 255) // 256 * 256, (dim + 63) // 64 * 64, 2 if dtype == 1 else 4
    copied = ld * es % 16 != 0
    weight = vocab * pitch * es
    bound = 400 << 20
    if es == 4:
        bound = max(bound, min(weight * 65 // 64, need(1, 152 * 256)))
    assert need(1, 0) <= max(bound, need(1, 4096) * 17 // 16 + (128 << 20))
    small = 40 * rows + (1 << 20)                 # labels, statistics and the like
    columns = 4096 * (rows + (pitch if copied else 0)) * es * 17 // 16
    columns = max(columns, (64 if es == 2 else 128) << 20)
    if copied:
        columns = max(columns, 390 << 20)
        if es == 4:
            columns = max(columns, min(weight, 152 * 256 * pitch * 4) + (128 << 20))
    assert need(0, 0) <= rows * pitch * es + small + columns * 65 // 64


@pytest.mark.parametrize("n,dim,vocab,tensor", [
    (1, 768, 50257, True), (1, 512, 128256, True), (1, 960, 50257, True), (2, 768, 128256, True),
    (2, 768, 50257, False), (1, 768, 32000, False), (1, 256, 250000, False),
    (1, 1024, 128256, False), (2, 4096, 128256, False), (3, 768, 8000, True)])
def test_head_loss_few_token_backward_follows_its_measurements(lib, n, dim, vocab, tensor):
    """Aligned bf16 rows: one pass over W (which needs the sums of 304 blocks only) or the tensor
    cores (which need pieces of G), whichever was faster at these sizes."""
    out = C.c_size_t(0)
    assert lib.mfsdp_head_loss_workspace_bytes(n, dim, vocab, 1, 1, P, dim, 0, C.byref(out)) == 0
    one_pass = 304 * n * dim * 4
    assert (out.value > 2 * one_pass + (2 << 20)) == tensor
    assert tensor or out.value <= one_pass + 1024


def test_binding_refuses_a_workspace_with_less_memory_than_elements():
    import torch

    from matrix_optimizer_owner_gb300 import mfsdp
    one = torch.empty(1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="contiguous"):
        mfsdp._workspace(one.expand(4096), 4096, one, one.get_device(), None, 0)
    ws = torch.empty(4096, dtype=torch.float32)
    assert mfsdp._workspace(ws, 4096, one, one.get_device(), None, 0) == (ws, 4 * 4096)


def test_kept_workspaces_are_bounded_and_can_be_released(monkeypatch):
    import torch

    from matrix_optimizer_owner_gb300 import mfsdp
    monkeypatch.setattr(mfsdp, "_is_capturing", lambda: False)
    monkeypatch.setattr(mfsdp, "_U8", torch.uint8)
    monkeypatch.setattr(mfsdp, "_scratch", mfsdp._Scratch())
    like, kept = torch.empty(1), mfsdp._scratch.buffers
    for stream in range(20):
        mfsdp._workspace(None, 100, like, 0, None, stream)
        assert (0, stream) in kept and len(kept) <= 8
    first = kept[(0, 19)][1]
    assert mfsdp._workspace(None, 100, like, 0, None, 19)[0] is first
    mfsdp._workspace(None, 2 << 20, like, 0, None, 12)       # a larger one replaces its own only
    assert len(kept) == 8 and kept[(0, 12)][0] == 2 << 20 and kept[(0, 19)][1] is first
    mfsdp.mfsdp_release_workspaces()
    assert not kept
