"""The binding's default workspaces: one per host thread and stream, fresh ones for captures and
for explicit streams, so that calls that overlap never share one."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _case(n, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(700, (n,), generator=gen, device="cuda")
    return ids, torch.randn(n, 128, generator=gen, device="cuda")


def _grad(ids, dy, out):
    from matrix_optimizer_owner_gb300 import mfsdp
    mfsdp.mfsdp_embedding_backward(ids, dy, 1.0, out)
    return out


def test_kept_per_stream_and_grown():
    from matrix_optimizer_owner_gb300 import mfsdp
    mfsdp._scratch.buffers.clear()                   # what earlier tests left
    out = torch.empty(700, 128, device="cuda")
    _grad(*_case(10, 0), out)
    raw = torch.cuda.current_stream().cuda_stream
    key = (torch.cuda.current_device(), raw)
    first = mfsdp._scratch.buffers[key][1]
    _grad(*_case(10, 0), out)
    assert mfsdp._scratch.buffers[key][1] is first
    _grad(*_case(60000, 0), out)                     # a larger one replaces it
    grown = mfsdp._scratch.buffers[key]
    assert grown[1] is not first and grown[0] > first.numel()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _grad(*_case(10, 0), torch.empty_like(out))
    assert mfsdp._scratch.buffers[(key[0], s.cuda_stream)][1] is not grown[1]
    torch.cuda.synchronize()


def test_capture_does_not_use_the_kept_one():
    from matrix_optimizer_owner_gb300 import mfsdp
    ids, dy = _case(3000, 1)
    want = _grad(ids, dy, torch.empty(700, 128, device="cuda")).clone()
    out = torch.zeros_like(want)
    kept = dict(mfsdp._scratch.buffers)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _grad(ids, dy, out)
    assert mfsdp._scratch.buffers == kept
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_threads_and_streams_at_the_same_time():
    torch.cuda.synchronize()
    cases = [_case(2000 + 500 * i, 2 + i) for i in range(4)]
    want = [_grad(ids, dy, torch.empty(700, 128, device="cuda")).clone() for ids, dy in cases]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        torch.cuda.set_device(0)
        # two threads share a stream, two have their own
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                got[i] = _grad(*cases[i], torch.empty(700, 128, device="cuda"))
        streams[i].synchronize()

    a, b, c = (torch.cuda.Stream() for _ in range(3))
    streams = [a, a, b, c]
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_explicit_stream_leaves_the_current_streams_memory_alone():
    """A temporary of the workspace's size is freed while kernels queued on the current stream still
    use it.  A call on another stream must not take its memory."""
    from matrix_optimizer_owner_gb300 import mfsdp
    torch.cuda.synchronize()
    ids, dy = _case(3000, 9)
    want = _grad(ids, dy, torch.empty(700, 128, device="cuda")).clone()
    nbytes = mfsdp.mfsdp_embedding_backward_workspace_bytes(700, 128, 3000)
    for handle in (False, True):
        out, seen = torch.zeros_like(want), torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        temp = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        temp.fill_(7)
        torch.cuda._sleep(50_000_000)                # some 25 ms
        seen.copy_(temp)
        del temp                                     # free for the current stream, not for others
        mfsdp.mfsdp_embedding_backward(ids, dy, 1.0, out,
                                       stream=s.cuda_stream if handle else s)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and bool((seen == 7).all())


def test_threads_with_few_token_heads_of_different_widths():
    """A kernel's shared-memory limit is shared by all host threads: a narrow call must not lower it
    between a wide call's setting and its launch.  (The C entry points, called back to back: the
    binding's own time between two calls would hide it.)"""
    from matrix_optimizer_owner_gb300 import _lib, mfsdp
    lib = _lib.load()

    def case(dim, seed):
        """Arguments of both calls, and the tensors they point to."""
        gen = torch.Generator(device="cuda").manual_seed(seed)
        h = torch.randn(4, dim, generator=gen, device="cuda")
        w = torch.randn(64, dim, generator=gen, device="cuda") / dim ** 0.5
        lab = torch.randint(64, (4,), generator=gen, device="cuda")
        loss, lse = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
        out = [loss, lse, torch.empty_like(h), torch.empty_like(w)]
        ws = [torch.empty(mfsdp.mfsdp_head_loss_workspace_bytes(4, dim, w, back),
                          dtype=torch.uint8, device="cuda") for back in (False, True)]
        st = torch.cuda.Stream()
        both = (4, dim, 64, mfsdp.DTYPE_F32, h.data_ptr(), dim, w.data_ptr(), dim, mfsdp.INDEX_I64,
                lab.data_ptr(), -100)
        fwd = both + (loss.data_ptr(), lse.data_ptr(), ws[0].data_ptr(), ws[0].numel(),
                      st.cuda_stream)
        bwd = both + (lse.data_ptr(), lse.data_ptr(), 0, out[2].data_ptr(), dim, out[3].data_ptr(),
                      dim, ws[1].data_ptr(), ws[1].numel(), st.cuda_stream)
        return fwd, bwd, out, (h, w, lab, ws, st)

    # backward at 6400 takes all that the path may use, at 1600 a quarter; forward at 12800 and 3400
    cases = [case(d, i) for i, d in enumerate((6400, 1600, 12800, 3400))]
    torch.cuda.synchronize()
    for fwd, bwd, _, _ in cases:
        assert lib.mfsdp_head_loss_forward(*fwd) == 0 and lib.mfsdp_head_loss_backward(*bwd) == 0
    torch.cuda.synchronize()
    want = [[t.clone() for t in c[2]] for c in cases]
    start, status = threading.Barrier(4), [set() for _ in range(4)]

    def work(i):
        torch.cuda.set_device(0)
        call, args = ((lib.mfsdp_head_loss_backward, cases[i][1]) if i < 2
                      else (lib.mfsdp_head_loss_forward, cases[i][0]))
        start.wait()
        for _ in range(5000):
            status[i].add(call(*args))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [{0}] * 4
    for (_, _, out, _), ref in zip(cases, want):
        assert all(torch.equal(x, y) for x, y in zip(out, ref))
