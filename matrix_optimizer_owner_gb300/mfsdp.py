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
from typing import Any, NamedTuple, Optional, Sequence, Tuple

from . import _lib
from ._lib import CostModel, Fp8Struct, GemmProblem, Matrix, ParamDesc, RankResources, Segment

POLICY_ROLE_GREEDY = 0
POLICY_SCOPE_GREEDY = 1
DTYPE_F32 = 0
DTYPE_BF16 = 1
INDEX_I32 = 0
INDEX_I64 = 1
NORM_LAYER = 0
NORM_RMS = 1
GROUPS_ROW = 0
GROUPS_COL = 1
GROUPS_TILE = 2
ACT_SWIGLU = 0
ACT_GELU = 1
FP8_E4M3 = 0
FP8_E5M2 = 1
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


# ------------------------------------------------------------------------------- 8-bit operators
class Fp8Matrix(NamedTuple):
    """An 8-bit matrix: ``data`` [rows, cols] of float8_e4m3fn or float8_e5m2 (16-byte aligned, rows a
    multiple of 16 bytes apart), ``scales`` of float8_e8m0fnu (or uint8), one per group of 128 values
    as ``groups`` (GROUPS_ROW, GROUPS_COL, GROUPS_TILE) says."""
    data: Any
    scales: Any
    groups: int


def fp8_scale_shape(rows: int, cols: int, groups: int) -> Tuple[int, int]:
    return (rows if groups == GROUPS_ROW else -(-rows // 128),
            cols if groups == GROUPS_COL else -(-cols // 128))


def fp8_empty(rows: int, cols: int, groups: int, dtype=None, device="cuda") -> Fp8Matrix:
    """An 8-bit matrix (of float8_e4m3fn unless ``dtype`` says otherwise) of uninitialised values."""
    import torch
    pitch = -(-cols // 16) * 16
    data = torch.empty((rows, pitch), dtype=dtype or torch.float8_e4m3fn, device=device)
    scales = torch.empty(fp8_scale_shape(rows, cols, groups), dtype=torch.float8_e8m0fnu,
                         device=device)
    return Fp8Matrix(data[:, :cols], scales, groups)


_FP8_CODES, _SCALE_TYPES = {}, ()
_GROUP_KINDS = (GROUPS_ROW, GROUPS_COL, GROUPS_TILE)


def _learn_fp8() -> None:
    global _SCALE_TYPES
    import torch
    _learn_dtypes()
    _FP8_CODES.update({torch.float8_e4m3fn: FP8_E4M3, torch.float8_e5m2: FP8_E5M2})
    _SCALE_TYPES = (torch.float8_e8m0fnu, torch.uint8)


def _fp8(m, shape, dev: int, name: str, groups: Optional[int] = None) -> Optional[Fp8Struct]:
    """The C description of an 8-bit matrix (None for None).  What a well-formed one needs is looked at
    in one go; anything else is sorted out by ``_fp8_checked``."""
    if m is None:
        return None
    data, scales, kind = m
    code = _FP8_CODES.get(data.dtype)
    rows, cols = shape
    ld, step = data.stride()
    ld_s, step_s = scales.stride()
    s_shape = (rows if kind == 0 else (rows + 127) >> 7, cols if kind == 1 else (cols + 127) >> 7)
    if (code is None or step != 1 or step_s != 1 or (groups is not None and kind != groups)
            or data.shape != shape or scales.shape != s_shape or data.get_device() != dev
            or scales.get_device() != dev or scales.dtype not in _SCALE_TYPES
            or kind not in _GROUP_KINDS):
        return _fp8_checked(m, shape, dev, name, groups)
    if rows < 2:                           # a single row has no pitch
        ld = (max(ld, cols) + 15) & -16
    if s_shape[0] < 2:
        ld_s = max(ld_s, s_shape[1])
    return Fp8Struct(data.data_ptr(), ld, scales.data_ptr(), ld_s, code, kind)


def _fp8_checked(m, shape, dev: int, name: str, groups: Optional[int]) -> Fp8Struct:
    data, scales, kind = m
    if not _FP8_CODES:
        _learn_fp8()
    code = _FP8_CODES.get(data.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float8_e4m3fn or float8_e5m2, got {data.dtype}")
    if kind not in _GROUP_KINDS:
        raise ValueError(f"{name}: unknown groups {kind}")
    if groups is not None and kind != groups:
        raise ValueError(f"{name}: expected groups {groups}, got {kind}")
    ld = _matrix(data, shape, data.dtype, dev, name)
    rows, cols = shape
    if rows <= 1:
        ld = (ld + 15) & -16
    if scales.dtype not in _SCALE_TYPES:
        raise TypeError(f"{name}: expected float8_e8m0fnu or uint8 scales, got {scales.dtype}")
    ld_s = _matrix(scales, fp8_scale_shape(rows, cols, kind), scales.dtype, dev, name + " scales")
    return Fp8Struct(data.data_ptr(), ld, scales.data_ptr(), ld_s, code, kind)


def mfsdp_quantize_fp8(x, out: Fp8Matrix, also: Optional[Fp8Matrix] = None, stream=None) -> None:
    """``x`` (float32 or bfloat16) in 8 bits: into ``out``, of any grouping, and from the same read
    into ``also``, a GROUPS_COL matrix beside a GROUPS_ROW one."""
    shape = _two_dims(x, "x")
    code, dev = _float_code(x, "x"), x.get_device()
    ld = _matrix(x, shape, x.dtype, dev, "x")
    o, a = _fp8(out, shape, dev, "out"), _fp8(also, shape, dev, "also")
    st = _device_stream(dev, stream)
    _check("mfsdp_quantize_fp8", _lib.load().mfsdp_quantize_fp8(
        shape[0], shape[1], code, x.data_ptr(), ld, o, a, st))


def mfsdp_regroup_fp8(src: Fp8Matrix, out: Fp8Matrix, also: Optional[Fp8Matrix] = None,
                      stream=None) -> None:
    """``src`` in another grouping (or type): what ``mfsdp_quantize_fp8`` gives for its values."""
    shape = _two_dims(src.data, "src")
    dev = src.data.get_device()
    s = _fp8(src, shape, dev, "src")
    o, a = _fp8(out, shape, dev, "out"), _fp8(also, shape, dev, "also")
    st = _device_stream(dev, stream)
    _check("mfsdp_regroup_fp8", _lib.load().mfsdp_regroup_fp8(shape[0], shape[1], s, o, a, st))


def mfsdp_dequantize_fp8(src: Fp8Matrix, out, stream=None) -> None:
    """The values of ``src`` into ``out`` (float32 or bfloat16)."""
    shape = _two_dims(src.data, "src")
    dev = src.data.get_device()
    s = _fp8(src, shape, dev, "src")
    code = _float_code(out, "out")
    ld = _matrix(out, shape, out.dtype, dev, "out")
    st = _device_stream(dev, stream)
    _check("mfsdp_dequantize_fp8", _lib.load().mfsdp_dequantize_fp8(
        shape[0], shape[1], s, code, out.data_ptr(), ld, st))


def mfsdp_gemm_fp8(a: Fp8Matrix, b: Fp8Matrix, c, trans_a: bool = False, trans_b: bool = False,
                   accumulate: bool = False, stream=None) -> None:
    """``c = op(a) @ op(b)`` of 8-bit matrices (op = transpose where ``trans_a`` / ``trans_b``), in
    float32 or bfloat16; added to ``c`` with ``accumulate``.  Scales are shared along the contraction:
    GROUPS_ROW or GROUPS_TILE for ``a`` and for ``b`` with ``trans_b``, GROUPS_COL or GROUPS_TILE for
    ``b`` and for ``a`` with ``trans_a``."""
    sa, sb = _two_dims(a.data, "a"), _two_dims(b.data, "b")
    m, k = (sa[1], sa[0]) if trans_a else (sa[0], sa[1])
    kb, n = (sb[1], sb[0]) if trans_b else (sb[0], sb[1])
    if kb != k:
        raise ValueError(f"a and b: contractions of {k} and {kb}")
    dev = c.get_device()
    code = _float_code(c, "c")
    ld = _matrix(c, (m, n), c.dtype, dev, "c")
    fa, fb = _fp8(a, sa, dev, "a"), _fp8(b, sb, dev, "b")
    st = _device_stream(dev, stream)
    _check("mfsdp_gemm_fp8", _lib.load().mfsdp_gemm_fp8(
        m, n, k, fa, 1 if trans_a else 0, fb, 1 if trans_b else 0, 1 if accumulate else 0, code,
        c.data_ptr(), ld, st))


def _rows(t, shape, dtype, dev: int, name: str):
    """Address and pitch of a 2D tensor that may be None."""
    if t is None:
        return None, shape[1]
    return t.data_ptr(), _matrix(t, shape, dtype, dev, name)


def mfsdp_norm_residual_forward(kind: int, x, residual, weight, bias, eps: float, h=None, y=None,
                                y8: Optional[Fp8Matrix] = None, h8: Optional[Fp8Matrix] = None,
                                mean=None, rstd=None, stream=None) -> None:
    """``h = x + residual`` (``residual`` may be None) and its layer or RMS norm into ``y``, into
    ``y8`` (8 bits, GROUPS_ROW), or both.  ``h`` (the residual stream), ``h8`` (its 8-bit checkpoint),
    ``mean`` and ``rstd`` are written where given, for ``mfsdp_norm_residual_backward``."""
    shape = _two_dims(x, "x")
    rows, cols = shape
    code, dtype, dev = _float_code(x, "x"), x.dtype, x.get_device()
    ld_x = _matrix(x, shape, dtype, dev, "x")
    rp, ld_r = _rows(residual, shape, dtype, dev, "residual")
    hp, ld_h = _rows(h, shape, dtype, dev, "h")
    yp, ld_y = _rows(y, shape, dtype, dev, "y")
    fy, fh = _fp8(y8, shape, dev, "y8", GROUPS_ROW), _fp8(h8, shape, dev, "h8", GROUPS_ROW)
    pdtype, pcode = _params_dtype(("weight", weight), ("bias", bias))
    w = _vector(weight, (cols,), pdtype, dev, "weight")
    b = _vector(bias, (cols,), pdtype, dev, "bias")
    m = _vector(mean, (rows,), _F32, dev, "mean")
    r = _vector(rstd, (rows,), _F32, dev, "rstd")
    st = _device_stream(dev, stream)
    _check("mfsdp_norm_residual_forward", _lib.load().mfsdp_norm_residual_forward(
        kind, rows, cols, code, pcode, x.data_ptr(), ld_x, rp, ld_r, w, b, eps, hp, ld_h, yp, ld_y,
        fy, fh, m, r, st))


def mfsdp_norm_residual_backward(kind: int, dy, dres, h, weight, mean, rstd, dx, dweight=None,
                                 dbias=None, workspace=None, stream=None) -> None:
    """Gradient of ``mfsdp_norm_residual_forward`` for its inputs into ``dx``, with ``dres`` (may be
    None), the gradient that reaches ``h`` beside the norm, added; and for the weight and the bias
    where given.  ``h`` is what the forward pass wrote: the tensor, or the ``Fp8Matrix`` checkpoint."""
    shape = _two_dims(dy, "dy")
    rows, cols = shape
    code, dtype, dev = _float_code(dy, "dy"), dy.dtype, dy.get_device()
    ld_dy = _matrix(dy, shape, dtype, dev, "dy")
    rp, ld_r = _rows(dres, shape, dtype, dev, "dres")
    kept = isinstance(h, Fp8Matrix)
    fh = _fp8(h, shape, dev, "h", GROUPS_ROW) if kept else None
    hp, ld_h = _rows(None if kept else h, shape, dtype, dev, "h")
    ld_dx = _matrix(dx, shape, dtype, dev, "dx")
    pdtype, pcode = _params_dtype(("weight", weight), ("dweight", dweight), ("dbias", dbias))
    w = _vector(weight, (cols,), pdtype, dev, "weight")
    dw = _vector(dweight, (cols,), pdtype, dev, "dweight")
    db = _vector(dbias, (cols,), pdtype, dev, "dbias")
    m = _vector(mean, (rows,), _F32, dev, "mean")
    r = _vector(rstd, (rows,), _F32, dev, "rstd")
    st = _device_stream(dev, stream)
    ws, nbytes = _workspace(workspace, mfsdp_norm_backward_workspace_bytes(rows, cols), dy, dev,
                            stream, st)
    _check("mfsdp_norm_residual_backward", _lib.load().mfsdp_norm_residual_backward(
        kind, rows, cols, code, pcode, dy.data_ptr(), ld_dy, rp, ld_r, hp, ld_h, fh, w, m, r,
        dx.data_ptr(), ld_dx, dw, db, ws.data_ptr(), nbytes, st))


def mfsdp_activation_forward(kind: int, gate, up, y=None, y8: Optional[Fp8Matrix] = None,
                             gate8: Optional[Fp8Matrix] = None, up8: Optional[Fp8Matrix] = None,
                             stream=None) -> None:
    """SwiGLU of ``gate`` and ``up`` (ACT_SWIGLU) or GELU of ``gate`` (ACT_GELU; ``up`` is None) into
    ``y``, into ``y8`` (8 bits, GROUPS_ROW), or both.  ``gate8`` and ``up8`` take the inputs in 8 bits
    (GROUPS_ROW) where given, for ``mfsdp_activation_backward``."""
    shape = _two_dims(gate, "gate")
    code, dtype, dev = _float_code(gate, "gate"), gate.dtype, gate.get_device()
    ld_g = _matrix(gate, shape, dtype, dev, "gate")
    up_p, ld_u = _rows(up, shape, dtype, dev, "up")
    yp, ld_y = _rows(y, shape, dtype, dev, "y")
    fy, fg, fu = (_fp8(m, shape, dev, name, GROUPS_ROW)
                  for m, name in ((y8, "y8"), (gate8, "gate8"), (up8, "up8")))
    st = _device_stream(dev, stream)
    _check("mfsdp_activation_forward", _lib.load().mfsdp_activation_forward(
        kind, shape[0], shape[1], code, gate.data_ptr(), ld_g, up_p, ld_u, yp, ld_y, fy, fg, fu, st))


def mfsdp_activation_backward(kind: int, dy, gate, up, dgate=None, dup=None,
                              dgate8: Optional[Fp8Matrix] = None, dup8: Optional[Fp8Matrix] = None,
                              dgate8_col: Optional[Fp8Matrix] = None,
                              dup8_col: Optional[Fp8Matrix] = None, stream=None) -> None:
    """Gradients of ``mfsdp_activation_forward`` for its inputs.  ``gate`` and ``up`` are the forward
    pass's tensors or its ``Fp8Matrix`` checkpoints (both the same).  Each gradient is written in
    ``dy``'s dtype (``dgate``, ``dup``), in 8 bits for the product with the weight (``dgate8``,
    ``dup8``, GROUPS_ROW) and for the weight's gradient (``dgate8_col``, ``dup8_col``, GROUPS_COL),
    wherever given."""
    shape = _two_dims(dy, "dy")
    code, dtype, dev = _float_code(dy, "dy"), dy.dtype, dy.get_device()
    ld_dy = _matrix(dy, shape, dtype, dev, "dy")
    args = []
    for t, name in ((gate, "gate"), (up, "up")):
        kept = isinstance(t, Fp8Matrix)
        args += [*_rows(None if kept else t, shape, dtype, dev, name),
                 _fp8(t, shape, dev, name, GROUPS_ROW) if kept else None]
    gp, ld_g = _rows(dgate, shape, dtype, dev, "dgate")
    up_p, ld_u = _rows(dup, shape, dtype, dev, "dup")
    fgr, fgc = _fp8(dgate8, shape, dev, "dgate8", GROUPS_ROW), _fp8(dgate8_col, shape, dev,
                                                                   "dgate8_col", GROUPS_COL)
    fur, fuc = _fp8(dup8, shape, dev, "dup8", GROUPS_ROW), _fp8(dup8_col, shape, dev, "dup8_col",
                                                               GROUPS_COL)
    st = _device_stream(dev, stream)
    _check("mfsdp_activation_backward", _lib.load().mfsdp_activation_backward(
        kind, shape[0], shape[1], code, dy.data_ptr(), ld_dy, *args, gp, ld_g, up_p, ld_u, fgr, fgc,
        fur, fuc, st))
