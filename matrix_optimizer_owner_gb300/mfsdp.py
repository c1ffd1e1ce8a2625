"""Python binding of ``include/mfsdp.h``: the same entry points, argument marshalling only.

Tensors are torch tensors on the current CUDA device (PyTorch provides device memory and
streams; every step of the optimizer runs in the library's kernels).  Each wrapper enqueues on
``torch.cuda.current_stream()`` unless a stream is given, and raises ``MfsdpError`` on a
non-zero status.
"""

from __future__ import annotations

import ctypes as C
import functools
import threading
from typing import Optional, Sequence, Tuple

from . import _lib
from ._lib import CostModel, GemmProblem, Matrix, ParamDesc, RankResources, Segment

POLICY_ROLE_GREEDY = 0
POLICY_SCOPE_GREEDY = 1
DTYPE_F32 = 0
DTYPE_BF16 = 1
INDEX_I32 = 0
INDEX_I64 = 1
NORM_LAYER = 0
NORM_RMS = 1
LR_ORIGINAL = 0
LR_MATCH_RMS_ADAMW = 1


class MfsdpError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {_lib.STATUS_NAMES.get(status, status)}")


def _check(fn: str, st: int) -> None:
    if st != 0:
        raise MfsdpError(fn, st)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:  # a tenth of the time of building a Stream object
            return raw(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _ptr_array(tensors: Sequence) -> C.Array:
    return (C.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"contribution dtype {t.dtype} is not float32 or bfloat16")


def mfsdp_version() -> int:
    return _lib.load().mfsdp_version()


def mfsdp_status_string(status: int) -> str:
    return _lib.load().mfsdp_status_string(status).decode()


# ------------------------------------------------------------------------------- planner
def mfsdp_plan_owner_set(params: Sequence[Tuple[int, int, int, bool]], world_size: int,
                         policy: int = POLICY_ROLE_GREEDY):
    """params: (rows, cols, block, is_matrix) per parameter, declaration order.

    Returns (segments, block_rank_numel, n_blocks): segments as a list of dicts with keys
    owner, role, local_offset, rank_offset, numel; block_rank_numel[k][r] = O_{B_k, r}.
    """
    lib = _lib.load()
    n = len(params)
    pd = (ParamDesc * max(n, 1))()
    for i, (r, c, b, m) in enumerate(params):
        pd[i] = ParamDesc(r, c, b, 1 if m else 0)
    seg = (Segment * max(n, 1))()
    brn = (C.c_int64 * max(n * world_size, 1))()
    nb = C.c_int64(0)
    _check("mfsdp_plan_owner_set",
           lib.mfsdp_plan_owner_set(pd, n, world_size, policy, seg, brn, C.byref(nb)))
    segs = [{"owner": s.owner, "role": s.role, "local_offset": s.local_offset,
             "rank_offset": s.rank_offset, "numel": s.numel} for s in seg[:n]]
    table = [[brn[k * world_size + r] for r in range(world_size)] for k in range(nb.value)]
    return segs, table, nb.value


def _param_array(params):
    n = len(params)
    pd = (ParamDesc * max(n, 1))()
    for i, (r, c, b, m) in enumerate(params):
        pd[i] = ParamDesc(r, c, b, 1 if m else 0)
    return pd


def _cost_model(param_bytes, grad_bytes, state_bytes, ns_steps):
    return CostModel(param_bytes, grad_bytes, state_bytes, ns_steps)


def mfsdp_score_plan(params: Sequence[Tuple[int, int, int, bool]], world_size: int,
                     segments: Sequence[dict], param_bytes: int = 2, grad_bytes: int = 2,
                     state_bytes: int = 4, ns_steps: int = 5):
    """Per-rank resource estimates and gamma_B of a plan (segments as returned by
    ``mfsdp_plan_owner_set``).  Returns (list of per-rank dicts, gamma per block)."""
    lib = _lib.load()
    n = len(params)
    seg = (Segment * max(n, 1))()
    for i, s in enumerate(segments):
        seg[i] = Segment(s["owner"], s["role"], s["local_offset"], s["rank_offset"], s["numel"])
    out = (RankResources * world_size)()
    gam = (C.c_double * max(n, 1))()
    nb = C.c_int64(0)
    model = _cost_model(param_bytes, grad_bytes, state_bytes, ns_steps)
    _check("mfsdp_score_plan", lib.mfsdp_score_plan(_param_array(params), n, world_size, seg,
                                                    C.byref(model), out, gam, C.byref(nb)))
    ranks = [{k: getattr(x, k) for k, _ in RankResources._fields_} for x in out]
    return ranks, [gam[k] for k in range(nb.value)]


def mfsdp_plan_cost_aware(params: Sequence[Tuple[int, int, int, bool]], world_size: int,
                          workspace_cap_bytes: int = 0, param_bytes: int = 2, grad_bytes: int = 2,
                          state_bytes: int = 4, ns_steps: int = 5):
    """CostAware plan.  Returns (segments, policy taken)."""
    lib = _lib.load()
    n = len(params)
    seg = (Segment * max(n, 1))()
    pol = C.c_int32(-1)
    model = _cost_model(param_bytes, grad_bytes, state_bytes, ns_steps)
    _check("mfsdp_plan_cost_aware",
           lib.mfsdp_plan_cost_aware(_param_array(params), n, world_size, C.byref(model),
                                     workspace_cap_bytes, seg, C.byref(pol)))
    segs = [{"owner": s.owner, "role": s.role, "local_offset": s.local_offset,
             "rank_offset": s.rank_offset, "numel": s.numel} for s in seg[:n]]
    return segs, pol.value


# ------------------------------------------------------------------------------- repacking
def _segment_array(segments):
    seg = (Segment * max(len(segments), 1))()
    for i, s in enumerate(segments):
        seg[i] = Segment(s["owner"], s["role"], s["local_offset"], s["rank_offset"], s["numel"])
    return seg


def mfsdp_repack_workspace_bytes(n_params: int) -> int:
    out = C.c_size_t(0)
    _check("mfsdp_repack_workspace_bytes",
           _lib.load().mfsdp_repack_workspace_bytes(n_params, C.byref(out)))
    return out.value


class RepackPlan:
    """A parameter list and its segment table marshalled once, for repeated pack / unpack
    calls (the per-call marshalling of a long list costs more host time than the copy)."""

    def __init__(self, params, segments, world_size: int):
        self.n = len(params)
        self.world_size = world_size
        self._pd = _param_array(params)
        self._seg = _segment_array(segments)

    def _ptrs(self, shards):
        return (C.c_void_p * self.world_size)(*[_ptr(t) for t in shards])

    def pack(self, canonical, shards, workspace, stream=None) -> None:
        _check("mfsdp_pack_owner_shards",
               _lib.load().mfsdp_pack_owner_shards(
                   self._pd, self.n, self._seg, self.world_size, canonical.element_size(),
                   _ptr(canonical), self._ptrs(shards), _ptr(workspace), workspace.numel(),
                   _stream(stream)))

    def unpack(self, shards, canonical, workspace, stream=None) -> None:
        _check("mfsdp_unpack_owner_shards",
               _lib.load().mfsdp_unpack_owner_shards(
                   self._pd, self.n, self._seg, self.world_size, canonical.element_size(),
                   self._ptrs(shards), _ptr(canonical), _ptr(workspace), workspace.numel(),
                   _stream(stream)))


def mfsdp_pack_owner_shards(params, segments, world_size: int, canonical, shards, workspace,
                            stream=None) -> None:
    """Canonical tensor -> owner shard tensors (``shards[r]`` may be None to skip rank r).
    All tensors share one element size; ``workspace`` is a uint8 device tensor."""
    eb = canonical.element_size()
    ptrs = (C.c_void_p * world_size)(*[_ptr(t) for t in shards])
    _check("mfsdp_pack_owner_shards",
           _lib.load().mfsdp_pack_owner_shards(_param_array(params), len(params),
                                               _segment_array(segments), world_size, eb,
                                               _ptr(canonical), ptrs, _ptr(workspace),
                                               workspace.numel(), _stream(stream)))


def mfsdp_unpack_owner_shards(params, segments, world_size: int, shards, canonical, workspace,
                              stream=None) -> None:
    """Owner shard tensors (None entries skipped) -> canonical tensor."""
    eb = canonical.element_size()
    ptrs = (C.c_void_p * world_size)(*[_ptr(t) for t in shards])
    _check("mfsdp_unpack_owner_shards",
           _lib.load().mfsdp_unpack_owner_shards(_param_array(params), len(params),
                                                 _segment_array(segments), world_size, eb, ptrs,
                                                 _ptr(canonical), _ptr(workspace),
                                                 workspace.numel(), _stream(stream)))


# ------------------------------------------------------------------------------- Shampoo
SHAMPOO_FP32 = 0
SHAMPOO_SPLIT_BF16 = 1

class ShampooSet:
    """Handle of ``mfsdp_shampoo_set``: the owned matrices of an owner Shampoo step."""

    def __init__(self, mats: Sequence[Tuple[int, int, int]]):
        lib = _lib.load()
        n = len(mats)
        arr = (Matrix * max(n, 1))()
        for i, (r, c, off) in enumerate(mats):
            arr[i] = Matrix(r, c, off)
        h = C.c_void_p()
        _check("mfsdp_shampoo_set_create", lib.mfsdp_shampoo_set_create(arr, n, C.byref(h)))
        self._h = h
        ws, ln, rn = C.c_size_t(0), C.c_int64(0), C.c_int64(0)
        _check("mfsdp_shampoo_set_sizes",
               lib.mfsdp_shampoo_set_sizes(h, C.byref(ws), C.byref(ln), C.byref(rn)))
        self.workspace_bytes, self.l_numel, self.r_numel = ws.value, ln.value, rn.value

    def close(self) -> None:
        if self._h:
            _lib.load().mfsdp_shampoo_set_destroy(self._h)
            self._h = None

    __del__ = close

    def init_state(self, eps: float, l, r, workspace, stream=None) -> None:
        _check("mfsdp_shampoo_init_state",
               _lib.load().mfsdp_shampoo_init_state(self._h, eps, _ptr(l), _ptr(r),
                                                    _ptr(workspace), workspace.numel(),
                                                    _stream(stream)))

    def step(self, grad, l, r, weights, lr: float, weight_decay: float, root_iters: int,
             workspace, stream=None, precision: int = 0) -> None:
        """``precision``: SHAMPOO_FP32 (CUDA-core fp32 products) or SHAMPOO_SPLIT_BF16 (root
        iteration and preconditioning on the tensor cores, split-bf16 operands)."""
        _check("mfsdp_shampoo_step",
               _lib.load().mfsdp_shampoo_step(self._h, _ptr(grad), _ptr(l), _ptr(r),
                                              _ptr(weights), lr, weight_decay, root_iters,
                                              precision, _ptr(workspace), workspace.numel(),
                                              _stream(stream)))


# ------------------------------------------------------------------------------- SOAP
class SoapSet:
    """Handle of ``mfsdp_soap_set``: the owned matrices of an owner SOAP step.  ``state``
    arguments are dicts of fp32 device tensors with the keys of ``SOAP_STATE_KEYS``."""

    SOAP_STATE_KEYS = ("l", "r", "q_l", "q_r", "eig_l", "eig_r", "exp_avg", "exp_avg_sq")

    def __init__(self, mats: Sequence[Tuple[int, int, int]]):
        lib = _lib.load()
        n = len(mats)
        arr = (Matrix * max(n, 1))()
        for i, (r, c, off) in enumerate(mats):
            arr[i] = Matrix(r, c, off)
        h = C.c_void_p()
        _check("mfsdp_soap_set_create", lib.mfsdp_soap_set_create(arr, n, C.byref(h)))
        self._h = h
        ws, ln, rn, el, er = (C.c_size_t(0), C.c_int64(0), C.c_int64(0), C.c_int64(0),
                              C.c_int64(0))
        _check("mfsdp_soap_set_sizes",
               lib.mfsdp_soap_set_sizes(h, C.byref(ws), C.byref(ln), C.byref(rn), C.byref(el),
                                        C.byref(er)))
        self.workspace_bytes = ws.value
        self.l_numel, self.r_numel = ln.value, rn.value
        self.eig_l_numel, self.eig_r_numel = el.value, er.value
        self.n_mats = n

    def close(self) -> None:
        if self._h:
            _lib.load().mfsdp_soap_set_destroy(self._h)
            self._h = None

    __del__ = close

    def state_sizes(self, numel: int):
        """numel of every state buffer for owner buffers of ``numel`` elements."""
        return {"l": self.l_numel, "r": self.r_numel, "q_l": self.l_numel,
                "q_r": self.r_numel, "eig_l": self.eig_l_numel, "eig_r": self.eig_r_numel,
                "exp_avg": numel, "exp_avg_sq": numel}

    @staticmethod
    def _state(state) -> "_lib.SoapState":
        return _lib.SoapState(*[_ptr(state[k]) for k in SoapSet.SOAP_STATE_KEYS])

    def init_state(self, state, workspace, stream=None) -> None:
        st = self._state(state)
        _check("mfsdp_soap_init_state",
               _lib.load().mfsdp_soap_init_state(self._h, C.byref(st), _ptr(workspace),
                                                 workspace.numel(), _stream(stream)))

    def step(self, grad, weights, state, t: int, *, lr: float, beta1: float, beta2: float,
             beta_stats: float, eps: float, weight_decay: float, max_sweeps: int, workspace,
             info=None, stream=None, jacobi_tol: float = 0.0, refresh: bool = True) -> None:
        """``refresh`` false keeps the state's eigenbases for this step (SOAP refreshes them
        every f steps)."""
        st = self._state(state)
        hy = _lib.SoapHyper(lr, beta1, beta2, beta_stats, eps, weight_decay, max_sweeps,
                            jacobi_tol, 1 if refresh else 0)
        _check("mfsdp_soap_step",
               _lib.load().mfsdp_soap_step(self._h, _ptr(grad), _ptr(weights), C.byref(st), t,
                                           C.byref(hy), _ptr(info) if info is not None else None,
                                           _ptr(workspace), workspace.numel(),
                                           _stream(stream)))


# ------------------------------------------------------------------------------- owner set
class OwnerSet:
    """Handle of ``mfsdp_owner_set``: create, query workspace, bind, destroy."""

    def __init__(self, mats: Sequence[Tuple[int, int, int]], split_max_numel: int = 0):
        lib = _lib.load()
        n = len(mats)
        arr = (Matrix * max(n, 1))()
        for i, (r, c, off) in enumerate(mats):
            arr[i] = Matrix(r, c, off)
        h = C.c_void_p()
        _check("mfsdp_owner_set_create",
               lib.mfsdp_owner_set_create(arr, n, split_max_numel, C.byref(h)))
        self.handle = h
        self.n_mats = n
        self._bound = ()

    def workspace_bytes(self) -> int:
        b = C.c_size_t(0)
        _check("mfsdp_owner_set_workspace_bytes",
               _lib.load().mfsdp_owner_set_workspace_bytes(self.handle, C.byref(b)))
        return b.value

    def split_count(self) -> int:
        k = C.c_int32(0)
        _check("mfsdp_owner_set_split_count",
               _lib.load().mfsdp_owner_set_split_count(self.handle, C.byref(k)))
        return k.value

    def bind(self, workspace, ns_input, ns_input_lo, ortho_out, ortho_lo, stream=None) -> None:
        _check("mfsdp_owner_set_bind", _lib.load().mfsdp_owner_set_bind(
            self.handle, _ptr(workspace), workspace.numel() * workspace.element_size(),
            _ptr(ns_input), _ptr(ns_input_lo), _ptr(ortho_out), _ptr(ortho_lo), _stream(stream)))
        self._bound = (workspace, ns_input, ns_input_lo, ortho_out, ortho_lo)  # keep alive

    def close(self) -> None:
        if self.handle:
            _lib.load().mfsdp_owner_set_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------------------- step calls
def mfsdp_owner_reduce_momentum(oset: OwnerSet, contrib: Sequence, grad_scale: float,
                                momentum: float, nesterov: bool, momentum_buf, ns_input,
                                ns_input_lo, reduced_grad_out, norm_out, stream=None) -> None:
    ptrs = _ptr_array(contrib)
    _check("mfsdp_owner_reduce_momentum", _lib.load().mfsdp_owner_reduce_momentum(
        oset.handle, ptrs, len(contrib), _dtype_code(contrib[0]), grad_scale, momentum,
        1 if nesterov else 0, _ptr(momentum_buf), _ptr(ns_input), _ptr(ns_input_lo),
        _ptr(reduced_grad_out), _ptr(norm_out), _stream(stream)))


def mfsdp_newton_schulz(oset: OwnerSet, ns_input, ns_input_lo, norm, steps: int, a: float,
                        b: float, c: float, eps: float, ortho_out, ortho_lo, stream=None) -> None:
    _check("mfsdp_newton_schulz", _lib.load().mfsdp_newton_schulz(
        oset.handle, _ptr(ns_input), _ptr(ns_input_lo), _ptr(norm), steps, a, b, c, eps,
        _ptr(ortho_out), _ptr(ortho_lo), _stream(stream)))


def mfsdp_apply_update(oset: OwnerSet, weights, ortho, ortho_lo, lr: float, weight_decay: float,
                       lr_adjust: int = LR_ORIGINAL, stream=None) -> None:
    _check("mfsdp_apply_update", _lib.load().mfsdp_apply_update(
        oset.handle, _ptr(weights), _ptr(ortho), _ptr(ortho_lo), lr, weight_decay, lr_adjust,
        _stream(stream)))


def mfsdp_adamw_tail(contrib: Sequence, grad_scale: float, param, exp_avg, exp_avg_sq, step: int,
                     lr: float, beta1: float, beta2: float, eps: float, weight_decay: float,
                     stream=None) -> None:
    ptrs = _ptr_array(contrib)
    _check("mfsdp_adamw_tail", _lib.load().mfsdp_adamw_tail(
        ptrs, len(contrib), _dtype_code(contrib[0]), grad_scale, param.numel(), _ptr(param),
        _ptr(exp_avg), _ptr(exp_avg_sq), step, lr, beta1, beta2, eps, weight_decay,
        _stream(stream)))


def mfsdp_query_status(stream=None) -> int:
    out = C.c_int32(0)
    _check("mfsdp_query_status", _lib.load().mfsdp_query_status(_stream(stream), C.byref(out)))
    return out.value


def mfsdp_set_wait_limit_ns(limit_ns: int) -> None:
    _check("mfsdp_set_wait_limit_ns", _lib.load().mfsdp_set_wait_limit_ns(limit_ns))


def mfsdp_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    _check("mfsdp_selftest_wait_timeout",
           _lib.load().mfsdp_selftest_wait_timeout(limit_ns, _stream(stream)))


def _fresh_workspace(nbytes: int, like, stream):
    """A uint8 workspace on `like`'s device from the pool of the stream the call runs on (None: the
    current one): whatever used that memory before, and whatever gets it next, is ordered with the
    call by that stream.  (The current stream's pool may hand out memory that kernels queued there
    still use.)"""
    import torch
    if stream is None:
        return like.new_empty((nbytes or 1,), dtype=torch.uint8)
    with torch.cuda.stream(stream if hasattr(stream, "cuda_stream")
                           else torch.cuda.ExternalStream(stream)):
        return like.new_empty((nbytes or 1,), dtype=torch.uint8)


# ------------------------------------------------------------------------------- fp32 GEMM
def mfsdp_gemm_f32_batched(problems, trans_a: bool = False, trans_b: bool = False,
                           workspace=None, stream=None) -> None:
    """C_i = alpha_i op(A_i) op(B_i) + beta_i C_i for every (A, B, C, alpha, beta) in
    ``problems`` (fp32 2D tensors on the current device, row-major with unit column stride);
    op = transpose where ``trans_a`` / ``trans_b``.  ``workspace`` (uint8 tensor) defaults
    to a fresh one of mfsdp_gemm_f32_workspace_bytes(len(problems)) bytes."""
    import torch
    lib = _lib.load()
    n = len(problems)
    tab = (GemmProblem * max(n, 1))()
    for i, (a, b, c, alpha, beta) in enumerate(problems):
        for t in (a, b, c):
            if t.dtype != torch.float32 or t.dim() != 2 or t.stride(1) != 1:
                raise TypeError("fp32 2D row-major tensors expected")
        m, k = (a.shape[1], a.shape[0]) if trans_a else (a.shape[0], a.shape[1])
        nn = b.shape[0] if trans_b else b.shape[1]
        tab[i] = GemmProblem(a.data_ptr(), b.data_ptr(), c.data_ptr(), m, nn, k, a.stride(0),
                             b.stride(0), c.stride(0), alpha, beta)
    if workspace is None:
        workspace = _fresh_workspace(lib.mfsdp_gemm_f32_workspace_bytes(n),
                                     problems[0][2] if n else torch.empty(0), stream)
    _check("mfsdp_gemm_f32_batched",
           lib.mfsdp_gemm_f32_batched(tab, n, 1 if trans_a else 0, 1 if trans_b else 0,
                                      _ptr(workspace), workspace.numel(), _stream(stream)))



# ------------------------------------------------------------------------------- operators
# A call on a small tensor is bound by the time spent here, so each tensor is checked in one
# helper call, by plain comparisons.
_FLOAT_CODES, _INDEX_CODES = {}, {}
_F32 = _U8 = _current_device = _current_raw_stream = _is_capturing = None


def _learn_dtypes() -> None:
    global _F32, _U8, _current_device, _current_raw_stream, _is_capturing
    import torch
    _F32, _U8 = torch.float32, torch.uint8
    _is_capturing = torch.cuda.is_current_stream_capturing
    _current_device = torch.cuda.current_device
    _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _FLOAT_CODES.update({torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16})
    _INDEX_CODES.update({torch.int32: INDEX_I32, torch.int64: INDEX_I64})


def _float_code(t, name: str) -> int:
    if _F32 is None:
        _learn_dtypes()
    code = _FLOAT_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float32 or bfloat16, got {t.dtype}")
    return code


def _index_code(t, name: str) -> int:
    if _F32 is None:
        _learn_dtypes()
    code = _INDEX_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected int32 or int64, got {t.dtype}")
    return code


def _refuse(t, shape, dtype, name: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if len(shape) == 2 or t.is_contiguous():
        raise ValueError(f"{name}: on {t.device}, expected tensors on the current CUDA device")
    raise ValueError(f"{name}: expected a contiguous vector, got strides {t.stride()}")


def _matrix(t, shape, dtype, dev: int, name: str) -> int:
    """Pitch of a 2D tensor of unit column stride."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, shape, dtype, name)
    pitch, step = t.stride()
    rows, cols = shape
    if step != 1 and cols > 1:
        raise ValueError(f"{name}: expected unit column stride, got strides {t.stride()}")
    return pitch if rows > 1 else max(pitch, cols)


def _vector(t, shape, dtype, dev: int, name: str) -> Optional[int]:
    """Address of a contiguous vector, or None."""
    if t is None:
        return None
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(t, shape, dtype, name)
    return t.data_ptr()


def _two_dims(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected two dimensions, got {tuple(t.shape)}")
    return t.shape


def _device_stream(dev: int, stream) -> Optional[int]:
    """The stream to launch on; `dev`, which holds every tensor, has to be the current CUDA
    device (a host pointer would fault the GPU)."""
    if dev < 0 or _current_device() != dev:
        raise ValueError("expected tensors on the current CUDA device")
    if stream is None and _current_raw_stream is not None:
        return _current_raw_stream(dev)
    return _stream(stream)


class _Scratch(threading.local):
    """The default workspaces of a host thread, one per device and stream.  Calls of one thread
    on one stream run in order, so they can share it; allocating one per call costs a small call
    half its time (a 768-wide norm's backward pass: 18 us of host time, 11 with a workspace).
    ``mfsdp_release_workspaces`` gives them back."""

    LIMIT = 64 << 20         # larger workspaces are not kept
    STREAMS = 8              # of more streams the one that came first loses its workspace

    def __init__(self):
        self.buffers = {}

    def get(self, nbytes: int, like, dev: int, raw: int):
        key = (dev, raw)
        size, buf = self.buffers.get(key, (0, None))
        if size < nbytes:
            size = max(nbytes, 1 << 20)
            buf = like.new_empty((size,), dtype=_U8)
            if key not in self.buffers and len(self.buffers) >= self.STREAMS:
                del self.buffers[next(iter(self.buffers))]
            self.buffers[key] = (size, buf)
        return buf


_scratch = _Scratch()


def mfsdp_release_workspaces() -> None:
    """Give the default workspaces that the calling thread's operator calls have kept back to
    PyTorch's allocator (at most 64 MiB for each of eight streams).  Calls still running on those
    streams are not disturbed: the memory stays ordered by its stream."""
    _scratch.buffers.clear()


def _workspace(ws, nbytes: int, like, dev: int, stream, raw: int):
    """The caller's uint8 workspace, or this thread's for the current stream.  A call on another
    stream, in a graph capture or with a large workspace gets a fresh one."""
    if ws is not None:
        if ws.get_device() != dev:
            raise ValueError("expected the workspace on the current CUDA device")
        if not ws.is_contiguous():       # an expanded tensor has less memory than elements
            raise ValueError(f"expected a contiguous workspace, got strides {ws.stride()}")
        return ws, ws.numel() * ws.element_size()
    if stream is None and nbytes <= _Scratch.LIMIT and not _is_capturing():
        return _scratch.get(nbytes, like, dev, raw), nbytes
    return _fresh_workspace(nbytes, like, stream), nbytes


def _params_dtype(*params):
    """The dtype of the first parameter vector there is (fp32 where there is none) and its
    code; the others are compared with it."""
    for name, t in params:
        if t is not None:
            return t.dtype, _float_code(t, name)
    return _F32, DTYPE_F32


def mfsdp_norm_forward(kind: int, x, weight, bias, eps: float, y, mean=None, rstd=None,
                       stream=None) -> None:
    """Layer norm (``kind`` NORM_LAYER) or RMS norm (NORM_RMS) of the rows of ``x`` into ``y``.
    ``weight`` and ``bias`` may be None; ``mean`` and ``rstd`` (fp32, per row) are written where
    given, for ``mfsdp_norm_backward``."""
    shape = _two_dims(x, "x")
    rows, cols = shape
    code, dtype, dev = _float_code(x, "x"), x.dtype, x.get_device()
    ld_x = _matrix(x, shape, dtype, dev, "x")
    ld_y = _matrix(y, shape, dtype, dev, "y")
    pdtype, pcode = _params_dtype(("weight", weight), ("bias", bias))
    w = _vector(weight, (cols,), pdtype, dev, "weight")
    b = _vector(bias, (cols,), pdtype, dev, "bias")
    m = _vector(mean, (rows,), _F32, dev, "mean")
    r = _vector(rstd, (rows,), _F32, dev, "rstd")
    st = _device_stream(dev, stream)
    _check("mfsdp_norm_forward", _lib.load().mfsdp_norm_forward(
        kind, rows, cols, code, pcode, x.data_ptr(), ld_x, w, b, eps, y.data_ptr(), ld_y, m, r,
        st))


@functools.lru_cache(maxsize=256)
def mfsdp_norm_backward_workspace_bytes(rows: int, cols: int) -> int:
    out = C.c_size_t(0)
    _check("mfsdp_norm_backward_workspace_bytes",
           _lib.load().mfsdp_norm_backward_workspace_bytes(rows, cols, C.byref(out)))
    return out.value


def mfsdp_norm_backward(kind: int, dy, x, weight, mean, rstd, dx, dweight=None, dbias=None,
                        workspace=None, stream=None) -> None:
    """Gradients of ``mfsdp_norm_forward`` for its input and, where given, for the weight and
    the bias.  ``workspace`` (uint8) defaults to this thread's for the current stream."""
    shape = _two_dims(x, "x")
    rows, cols = shape
    code, dtype, dev = _float_code(x, "x"), x.dtype, x.get_device()
    ld_x = _matrix(x, shape, dtype, dev, "x")
    ld_dy = _matrix(dy, shape, dtype, dev, "dy")
    ld_dx = _matrix(dx, shape, dtype, dev, "dx")
    pdtype, pcode = _params_dtype(("weight", weight), ("dweight", dweight), ("dbias", dbias))
    w = _vector(weight, (cols,), pdtype, dev, "weight")
    dw = _vector(dweight, (cols,), pdtype, dev, "dweight")
    db = _vector(dbias, (cols,), pdtype, dev, "dbias")
    m = _vector(mean, (rows,), _F32, dev, "mean")
    r = _vector(rstd, (rows,), _F32, dev, "rstd")
    st = _device_stream(dev, stream)
    ws, nbytes = _workspace(workspace, mfsdp_norm_backward_workspace_bytes(rows, cols), x, dev,
                            stream, st)
    _check("mfsdp_norm_backward", _lib.load().mfsdp_norm_backward(
        kind, rows, cols, code, pcode, dy.data_ptr(), ld_dy, x.data_ptr(), ld_x, w, m, r,
        dx.data_ptr(), ld_dx, dw, db, ws.data_ptr(), nbytes, st))


def mfsdp_embedding_forward(table, ids, scale: float, out, stream=None) -> None:
    """``out[t] = scale * table[ids[t]]``; the table and the output may differ in dtype."""
    shape = _two_dims(table, "table")
    vocab, dim = shape
    n, dev = ids.numel(), table.get_device()
    tcode, ocode = _float_code(table, "table"), _float_code(out, "out")
    icode = _index_code(ids, "ids")
    idp = _vector(ids, (n,), ids.dtype, dev, "ids")
    ld_t = _matrix(table, shape, table.dtype, dev, "table")
    ld_o = _matrix(out, (n, dim), out.dtype, dev, "out")
    st = _device_stream(dev, stream)
    _check("mfsdp_embedding_forward", _lib.load().mfsdp_embedding_forward(
        vocab, dim, tcode, table.data_ptr(), ld_t, n, icode, idp, scale, ocode, out.data_ptr(),
        ld_o, st))


@functools.lru_cache(maxsize=256)
def mfsdp_embedding_backward_workspace_bytes(vocab: int, dim: int, n_tokens: int) -> int:
    out = C.c_size_t(0)
    _check("mfsdp_embedding_backward_workspace_bytes",
           _lib.load().mfsdp_embedding_backward_workspace_bytes(vocab, dim, n_tokens,
                                                                C.byref(out)))
    return out.value


def mfsdp_embedding_backward(ids, dy, scale: float, dtable, padding_idx: int = -1,
                             accumulate: bool = False, workspace=None, stream=None) -> None:
    """Gradient of the table of ``mfsdp_embedding_forward``: overwrites ``dtable``, or adds to
    it with ``accumulate``.  Tokens of ``padding_idx`` take no part.  ``workspace`` (uint8)
    defaults to this thread's for the current stream."""
    shape = _two_dims(dtable, "dtable")
    vocab, dim = shape
    n, dev = ids.numel(), dtable.get_device()
    dcode, gcode = _float_code(dy, "dy"), _float_code(dtable, "dtable")
    icode = _index_code(ids, "ids")
    idp = _vector(ids, (n,), ids.dtype, dev, "ids")
    ld_dy = _matrix(dy, (n, dim), dy.dtype, dev, "dy")
    ld_dt = _matrix(dtable, shape, dtable.dtype, dev, "dtable")
    st = _device_stream(dev, stream)
    ws, nbytes = _workspace(workspace, mfsdp_embedding_backward_workspace_bytes(vocab, dim, n),
                            dtable, dev, stream, st)
    _check("mfsdp_embedding_backward", _lib.load().mfsdp_embedding_backward(
        vocab, dim, n, icode, idp, padding_idx, scale, dcode, dy.data_ptr(), ld_dy,
        1 if accumulate else 0, gcode, dtable.data_ptr(), ld_dt, ws.data_ptr(), nbytes, st))


@functools.lru_cache(maxsize=256)
def _head_workspace(n, dim, vocab, code, backward, misaligned, ld_w, piece) -> int:
    out = C.c_size_t(0)
    _check("mfsdp_head_loss_workspace_bytes", _lib.load().mfsdp_head_loss_workspace_bytes(
        n, dim, vocab, code, backward, misaligned, ld_w, piece, C.byref(out)))
    return out.value


def mfsdp_head_loss_workspace_bytes(n_tokens: int, dim: int, weight, backward: bool,
                                    piece: int = 0) -> int:
    vocab = weight.shape[0]
    ld_w = _matrix(weight, (vocab, dim), weight.dtype, weight.get_device(), "weight")
    return _head_workspace(n_tokens, dim, vocab, _float_code(weight, "weight"),
                           1 if backward else 0, weight.data_ptr() % 16, ld_w, piece)


def _head_args(hidden, weight, labels):
    shape = _two_dims(hidden, "hidden")
    n, dim = shape
    vocab = _two_dims(weight, "weight")[0]
    code, dtype, dev = _float_code(hidden, "hidden"), hidden.dtype, hidden.get_device()
    icode = _index_code(labels, "labels")
    lab = _vector(labels, (n,), labels.dtype, dev, "labels")
    ld_h = _matrix(hidden, shape, dtype, dev, "hidden")
    ld_w = _matrix(weight, (vocab, dim), dtype, dev, "weight")
    return n, dim, vocab, code, dtype, dev, icode, lab, ld_h, ld_w


def mfsdp_head_loss_forward(hidden, weight, labels, loss, lse, ignore_index: int = -100,
                            workspace=None, stream=None) -> None:
    """Per-token softmax cross entropy of ``hidden @ weight.T`` against ``labels`` into ``loss``
    and the log-sum-exp of the logits into ``lse`` (fp32, either may be None).  Tokens labelled
    ``ignore_index`` get 0 in both.  ``workspace`` (uint8) defaults to this thread's for the
    current stream."""
    n, dim, vocab, code, _, dev, icode, lab, ld_h, ld_w = _head_args(hidden, weight, labels)
    los = _vector(loss, (n,), _F32, dev, "loss")
    ls = _vector(lse, (n,), _F32, dev, "lse")
    st = _device_stream(dev, stream)
    wp = weight.data_ptr()
    ws, nbytes = _workspace(workspace, _head_workspace(n, dim, vocab, code, 0, wp % 16, ld_w, 0),
                            hidden, dev, stream, st)
    _check("mfsdp_head_loss_forward", _lib.load().mfsdp_head_loss_forward(
        n, dim, vocab, code, hidden.data_ptr(), ld_h, wp, ld_w, icode, lab, ignore_index, los, ls,
        ws.data_ptr(), nbytes, st))


def mfsdp_head_loss_backward(hidden, weight, labels, lse, dloss, dhidden=None, dweight=None,
                             ignore_index: int = -100, piece: int = 0, workspace=None,
                             stream=None) -> None:
    """Gradients of ``sum(dloss * loss)`` for the hidden states and the weight (either may be
    None), with ``lse`` from the forward pass; the logits are recomputed in pieces of ``piece``
    columns of the vocabulary (0: chosen)."""
    n, dim, vocab, code, dtype, dev, icode, lab, ld_h, ld_w = _head_args(hidden, weight, labels)
    ls = _vector(lse, (n,), _F32, dev, "lse")
    dl = _vector(dloss, (n,), _F32, dev, "dloss")
    ld_dh = ld_dw = dim
    dh = dw = None
    if dhidden is not None:
        ld_dh, dh = _matrix(dhidden, (n, dim), dtype, dev, "dhidden"), dhidden.data_ptr()
    if dweight is not None:
        ld_dw, dw = _matrix(dweight, (vocab, dim), dtype, dev, "dweight"), dweight.data_ptr()
    st = _device_stream(dev, stream)
    wp = weight.data_ptr()
    ws, nbytes = _workspace(workspace,
                            _head_workspace(n, dim, vocab, code, 1, wp % 16, ld_w, piece),
                            hidden, dev, stream, st)
    _check("mfsdp_head_loss_backward", _lib.load().mfsdp_head_loss_backward(
        n, dim, vocab, code, hidden.data_ptr(), ld_h, wp, ld_w, icode, lab, ignore_index, ls, dl,
        piece, dh, ld_dh, dw, ld_dw, ws.data_ptr(), nbytes, st))
