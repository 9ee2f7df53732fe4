"""ctypes binding to libasv.so: argument marshalling only (pointers, sizes, stream)."""
from __future__ import annotations

import ctypes as C
import functools
import importlib.machinery
import importlib.util
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

from . import nvcc_build as _build

ASV_F32 = 0
ASV_BF16 = 1
ASV_F16 = 2  # paged cache only
ASV_MODE_ASYMSPEC = 0
ASV_MODE_RAPID = 1
ASV_MODE_SCI = 2
REQ_NONFINITE = 1
REQ_BAD_DRAFT = 2
REQ_TIMEOUT = 4
REQ_BAD_PAGE = 8
REQ_BAD_LEN = 16

_STATUS = {0: "ASV_OK", 1: "ASV_ERR_NULL", 2: "ASV_ERR_SHAPE", 3: "ASV_ERR_ALIGN", 4: "ASV_ERR_DTYPE",
           5: "ASV_ERR_PARAM", 6: "ASV_ERR_WORKSPACE", 7: "ASV_ERR_CUDA"}


class AsvError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_lib = None
_lib_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def library():
    """Load libasv.so (raises if it has not been built)."""
    global _lib
    with _lib_lock:
        if _lib is None:
            if not os.path.exists(_build.LIB):
                raise AsvError(-1, f"libasv.so not built ({_build.LIB}); call speculative_decoding_logit_gb300.build()")
            lib = C.CDLL(_build.LIB)
            _declare(lib)
            _lib = lib
    return _lib


_vp = C.c_void_p
_i = C.c_int
_sz = C.c_size_t
_f = C.c_float


class _AsymOptionsC(C.Structure):
    _fields_ = [("delta_source", C.c_int)]


DELTA_A_MINUS_B = 0
DELTA_A = 1
DELTA_T_MINUS_B = 2


class _RapidOptionsC(C.Structure):
    _fields_ = [("tail_mode", C.c_int)]


class _SciStabC(C.Structure):
    _fields_ = [("hysteresis", C.c_double), ("min_refresh", C.c_int32), ("reserved", C.c_int32),
                ("fallback_acc", C.c_double), ("fallback_T", C.c_double)]


class _SciParamsC(C.Structure):
    _fields_ = [("T_base", C.c_double), ("alpha_omega", C.c_double), ("tau_credit", C.c_double),
                ("T_min", C.c_double), ("T_max", C.c_double), ("ewma_beta", C.c_double)]


class _PagedCacheC(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("dtype", C.c_int), ("num_pages", C.c_int),
                ("page_size", C.c_int), ("kv_heads", C.c_int), ("head_dim", C.c_int)] + [
                    (f"{t}_stride_{d}", C.c_int64) for t in "kv" for d in ("page", "slot", "head")]


class _PagedBatchC(C.Structure):
    _fields_ = [("B", C.c_int), ("N", C.c_int), ("indptr", C.c_void_p), ("cache_len", C.c_void_p),
                ("block_table", C.c_void_p), ("max_pages", C.c_int), ("block_table_stride", C.c_int64)]


class _RowsC(C.Structure):
    _fields_ = [("data", C.c_void_p), ("stride_token", C.c_int64), ("stride_head", C.c_int64)]


class _RotaryC(C.Structure):
    _fields_ = [("table", C.c_void_p), ("dim", C.c_int), ("max_position", C.c_int), ("interleaved", C.c_int)]


def _declare(L):
    L.asv_status_string.argtypes = [_i]
    L.asv_status_string.restype = C.c_char_p
    L.asv_last_cuda_error.argtypes = []
    L.asv_last_cuda_error.restype = _i
    L.asv_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
    L.asv_workspace_bytes.restype = _sz
    L.asv_workspace_init.argtypes = [_vp, _sz, _vp]
    L.asv_workspace_init.restype = _i
    L.asv_set_tuning.argtypes = [_i, _i]
    L.asv_set_tuning.restype = _i
    L.asv_set_kernel.argtypes = [_i]
    L.asv_set_kernel.restype = _i
    L.asv_query_plan.argtypes = [_i, _i, _i, _i, _i] + [C.POINTER(_i)] * 5
    L.asv_query_plan.restype = _i
    L.asymspec_verify.argtypes = [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _f, _f, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.asymspec_verify.restype = _i
    L.asymspec_verify_ex.argtypes = [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _f, _f, C.POINTER(_AsymOptionsC), _vp, _vp,
                                     _vp, _vp, _vp, _vp, _sz, _vp]
    L.asymspec_verify_ex.restype = _i
    L.asv_host_arena_bytes.argtypes = [_i, _i, _i, _i]
    L.asv_host_arena_bytes.restype = _sz
    L.asymspec_verify_host.argtypes = [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _f, _f, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.asymspec_verify_host.restype = _i
    L.rapid_verify.argtypes = [_vp, _vp, _vp, _i, _i, _i, _f, _f, _f, C.c_uint64, C.c_uint32, _vp, _vp, _vp, _vp,
                               _sz, _vp]
    L.rapid_verify.restype = _i
    L.sci_verify.argtypes = [_vp, _vp, _i, _vp, _i, _i, _i, C.POINTER(_SciParamsC), _vp, _vp, _vp, _vp, _vp, _vp,
                             _vp, _sz, _vp]
    L.sci_verify.restype = _i
    L.asymspec_verify_sweep.argtypes = [_vp, _vp, _vp, _i, _vp, _i, _i, _i, C.POINTER(_f), _i, C.POINTER(_f), _i,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.asymspec_verify_sweep.restype = _i
    L.asymspec_sci_verify.argtypes = [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _f, _f, C.POINTER(_SciParamsC), _vp, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.asymspec_sci_verify.restype = _i
    L.sci_verify_prehit.argtypes = [_vp, _vp, _i, _vp, _i, _i, _i, C.POINTER(_SciParamsC), _vp, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _sz, _vp]
    L.sci_verify_prehit.restype = _i
    L.rapid_verify_ex.argtypes = [_vp, _vp, _vp, _i, _i, _i, _f, _f, _f, C.c_uint64, C.c_uint32,
                                  C.POINTER(_RapidOptionsC), _vp, _vp, _vp, _vp, _sz, _vp]
    L.rapid_verify_ex.restype = _i
    L.sci_verify_ex.argtypes = [_vp, _vp, _i, _vp, _i, _i, _i, C.POINTER(_SciParamsC), C.POINTER(_SciStabC), _vp,
                                _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.sci_verify_ex.restype = _i
    L.paged_kv_append.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp]
    L.paged_kv_append.restype = _i
    L.asv_paged_workspace_bytes.argtypes = [_i, _i, _i]
    L.asv_paged_workspace_bytes.restype = _sz
    L.paged_attention.argtypes = [_vp, _vp, _vp, _vp, _i, _f, _i, _vp, _vp, _vp, _sz, _vp]
    L.paged_attention.restype = _i


def _check(status: int, what: str):
    if status != 0:
        L = library()
        msg = L.asv_status_string(status).decode()
        if status == 7:
            msg += f" (cudaError {L.asv_last_cuda_error()})"
        raise AsvError(status, f"{what}: {msg}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream_handle(device: torch.device, stream=None):
    if stream is not None and stream.device != device:
        raise AsvError(2, "the stream must be one of the tensors' device")
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _mark_used(tensors, caller):
    """Keeps the memory of a call's outputs from reuse until the caller's stream, which reads them, is done too."""
    for t in tensors:
        if t is not None:
            t.record_stream(caller)


def _made_on(stream, make):
    """The tensors that make() allocates for a call on `stream` (None: the current one).  They are made there, so
    that a zero-fill comes before the call and no block is taken that work on another stream still uses."""
    if stream is None:
        return make()
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        made = make()
    _mark_used(made, caller)
    return made


def _in_place(call):
    """`call` with its first argument's device current, where the launch goes, and with its `stream` current, so that
    its outputs and a new workspace are made there (see _made_on)."""
    @functools.wraps(call)
    def placed(*args, stream=None, **kw):
        first = args[0] if args else next(iter(kw.values()), None)
        if isinstance(first, torch.Tensor) and first.is_cuda and first.get_device() != torch._C._cuda_getDevice():
            with torch.cuda.device(first.device):
                return placed(*args, stream=stream, **kw)
        if stream is None:
            return call(*args, **kw)
        caller = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            got = call(*args, stream=stream, **kw)
        if kw.get("out") is None:
            _mark_used(vars(got).values(), caller)
        return got
    return placed


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return ASV_F32
    if t.dtype == torch.bfloat16:
        return ASV_BF16
    raise AsvError(4, f"logits must be float32 or bfloat16, got {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise AsvError(-1, "inputs must be CUDA tensors (the library has no CPU path)")


def _contig(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_contiguous():
        raise AsvError(2, f"{name} must be contiguous")
    return t


# Workspace cache: one zero-initialised buffer per (device, stream); every call leaves it zeroed.  One made
# while the stream is capturing belongs to the graph, whose replays zero-fill it, and is not kept.
_ws_cache: dict = {}
_ws_lock = threading.Lock()


def _workspace(device: torch.device, stream_handle: int, nbytes: int) -> torch.Tensor:
    key = (device.index, stream_handle)
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = torch.zeros(max(nbytes, 4096), dtype=torch.uint8, device=device)
            if not torch.cuda.is_current_stream_capturing():
                _ws_cache[key] = ws
    return ws


def workspace_bytes(mode: int, B: int, K: int, V: int, dtype: int) -> int:
    return int(library().asv_workspace_bytes(mode, B, K, V, dtype))


def set_tuning(cluster_ctas: int = 0, threads_per_cta: int = 0):
    _check(library().asv_set_tuning(cluster_ctas, threads_per_cta), "asv_set_tuning")


KERNEL_DEFAULT = 0
KERNEL_CLUSTER = 1
KERNEL_STAGED = 2


def set_kernel(which: int):
    """Kernel for later AsymSpec / E2-SCI calls: KERNEL_DEFAULT / KERNEL_CLUSTER (the cluster
    kernel) or KERNEL_STAGED (the staged kernel, where it applies)."""
    _check(library().asv_set_kernel(int(which)), "asv_set_kernel")


def query_plan(mode: int, B: int, K: int, V: int, dtype: int) -> dict:
    out = [C.c_int(0) for _ in range(5)]
    _check(library().asv_query_plan(mode, B, K, V, dtype, *[C.byref(o) for o in out]), "asv_query_plan")
    return {"cluster": out[0].value, "threads": out[1].value, "smem": out[2].value, "bulk": out[3].value,
            "max_active_clusters": out[4].value}


# ------------------------------------------------------------------ AsymSpec

@dataclass
class AsymSpecOutput:
    accept_len: torch.Tensor   # [B] int32
    tokens: torch.Tensor       # [B, K+1] int32, -1 padded
    D: torch.Tensor            # [B, K+1] float32
    lse: torch.Tensor          # [B, K+1, 3] float32 (a, b, t)
    req_status: torch.Tensor   # [B] int32 (ASV_REQ_* bits)


@_in_place
def asymspec_verify(a: torch.Tensor, b: torch.Tensor, t: torch.Tensor, draft_ids: torch.Tensor,
                    beta: float = 1.0, gamma: float = 0.5, *, delta_source: int = DELTA_A_MINUS_B,
                    out: Optional[AsymSpecOutput] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> AsymSpecOutput:
    """AsymSpec verification of a [B, K+1, V] batch (see include/asv.h).  `delta_source`
    selects the context-gain signal of the delta-fusion score (asymspec_verify_ex)."""
    _need_cuda(a, b, t, draft_ids)
    if a.dim() != 3 or a.shape != b.shape or a.shape != t.shape:
        raise AsvError(2, "a, b, t must share one [B, K+1, V] shape")
    if a.dtype != b.dtype or a.dtype != t.dtype:
        raise AsvError(4, "a, b, t must share one dtype")
    B, R1, V = a.shape
    K = R1 - 1
    if draft_ids.dtype != torch.int32 or tuple(draft_ids.shape) != (B, K):
        raise AsvError(2, "draft_ids must be int32 [B, K]")
    for n, x in (("a", a), ("b", b), ("t", t), ("draft_ids", draft_ids)):
        _contig(x, n)
    dev = a.device
    sh = _stream_handle(dev, stream)
    if out is None:
        out = AsymSpecOutput(torch.empty(B, dtype=torch.int32, device=dev),
                             torch.empty(B, R1, dtype=torch.int32, device=dev),
                             torch.empty(B, R1, dtype=torch.float32, device=dev),
                             torch.empty(B, R1, 3, dtype=torch.float32, device=dev),
                             torch.empty(B, dtype=torch.int32, device=dev))
    dt = _dtype_code(a)
    need = workspace_bytes(ASV_MODE_ASYMSPEC, B, K, V, dt)
    ws = workspace if workspace is not None else _workspace(dev, sh, need)
    if delta_source == DELTA_A_MINUS_B:
        st = library().asymspec_verify(_ptr(a), _ptr(b), _ptr(t), dt, _ptr(draft_ids), B, K, V, float(beta),
                                       float(gamma), _ptr(out.accept_len), _ptr(out.tokens), _ptr(out.D),
                                       _ptr(out.lse), _ptr(out.req_status), _ptr(ws), ws.numel() * ws.element_size(),
                                       sh)
        _check(st, "asymspec_verify")
    else:
        opt = _AsymOptionsC(int(delta_source))
        st = library().asymspec_verify_ex(_ptr(a), _ptr(b), _ptr(t), dt, _ptr(draft_ids), B, K, V, float(beta),
                                          float(gamma), C.byref(opt), _ptr(out.accept_len), _ptr(out.tokens),
                                          _ptr(out.D), _ptr(out.lse), _ptr(out.req_status), _ptr(ws),
                                          ws.numel() * ws.element_size(), sh)
        _check(st, "asymspec_verify_ex")
    return out


def host_arena_bytes(B: int, K: int, V: int, dtype: int) -> int:
    return int(library().asv_host_arena_bytes(B, K, V, dtype))


ASV_MODE_SWEEP = 3
ASV_MODE_ASYMSPEC_SCI = 4


@dataclass
class SweepOutput:
    accept_len: torch.Tensor  # [n_gamma, B] int32
    tokens: torch.Tensor      # [n_beta, n_gamma, B, K+1] int32
    D: torch.Tensor           # [B, K+1] float32
    lse: torch.Tensor         # [B, K+1, 3] float32
    req_status: torch.Tensor  # [B] int32


def _check_asym_inputs(a, b, t, draft_ids):
    _need_cuda(a, b, t, draft_ids)
    if a.dim() != 3 or a.shape != b.shape or a.shape != t.shape:
        raise AsvError(2, "a, b, t must share one [B, K+1, V] shape")
    if a.dtype != b.dtype or a.dtype != t.dtype:
        raise AsvError(4, "a, b, t must share one dtype")
    B, R1, V = a.shape
    if draft_ids.dtype != torch.int32 or tuple(draft_ids.shape) != (B, R1 - 1):
        raise AsvError(2, "draft_ids must be int32 [B, K]")
    for n, x in (("a", a), ("b", b), ("t", t), ("draft_ids", draft_ids)):
        _contig(x, n)
    return B, R1 - 1, V


@_in_place
def asymspec_verify_sweep(a: torch.Tensor, b: torch.Tensor, t: torch.Tensor, draft_ids: torch.Tensor, betas,
                          gammas, *, workspace: Optional[torch.Tensor] = None, stream=None) -> SweepOutput:
    """AsymSpec for every (beta, gamma) of a grid from one read of a, b, t (asymspec_verify_sweep)."""
    B, K, V = _check_asym_inputs(a, b, t, draft_ids)
    betas = [float(x) for x in betas]
    gammas = [float(x) for x in gammas]
    nb, ng = len(betas), len(gammas)
    dev = a.device
    sh = _stream_handle(dev, stream)
    out = SweepOutput(torch.empty(ng, B, dtype=torch.int32, device=dev),
                      torch.empty(nb, ng, B, K + 1, dtype=torch.int32, device=dev),
                      torch.empty(B, K + 1, dtype=torch.float32, device=dev),
                      torch.empty(B, K + 1, 3, dtype=torch.float32, device=dev),
                      torch.empty(B, dtype=torch.int32, device=dev))
    dt = _dtype_code(a)
    ws = workspace if workspace is not None else _workspace(dev, sh, workspace_bytes(ASV_MODE_SWEEP, B, K, V, dt))
    bb = (_f * max(nb, 1))(*betas)
    gg = (_f * max(ng, 1))(*gammas)
    st = library().asymspec_verify_sweep(_ptr(a), _ptr(b), _ptr(t), dt, _ptr(draft_ids), B, K, V, bb, nb, gg, ng,
                                         _ptr(out.accept_len), _ptr(out.tokens), _ptr(out.D), _ptr(out.lse),
                                         _ptr(out.req_status), _ptr(ws), ws.numel(), sh)
    _check(st, "asymspec_verify_sweep")
    return out


@dataclass
class AsymSciOutput:
    accept_len: torch.Tensor      # AsymSpec [B]
    tokens: torch.Tensor          # AsymSpec [B, K+1]
    D: torch.Tensor               # JSD(a || b) [B, K+1]
    lse: torch.Tensor             # [B, K+1, 3]
    sci_accept_len: torch.Tensor  # E2-SCI [B]
    sci_tokens: torch.Tensor      # E2-SCI [B, K+1]
    jsd: torch.Tensor             # JSD(a || t) [B, K+1]
    T: torch.Tensor               # E2-SCI threshold [B]
    req_status: torch.Tensor      # [B]


@_in_place
def asymspec_sci_verify(a: torch.Tensor, b: torch.Tensor, t: torch.Tensor, draft_ids: torch.Tensor, beta: float,
                        gamma: float, r_hat: torch.Tensor, params: "SciParams" = None, *,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> AsymSciOutput:
    """AsymSpec and one E2-SCI window (draft = a, target = t) from one read (asymspec_sci_verify);
    r_hat (float64 [B], device) is updated in place."""
    B, K, V = _check_asym_inputs(a, b, t, draft_ids)
    if r_hat.dtype != torch.float64 or tuple(r_hat.shape) != (B,) or not r_hat.is_cuda:
        raise AsvError(2, "r_hat must be a float64 [B] CUDA tensor")
    params = params or SciParams()
    dev = a.device
    sh = _stream_handle(dev, stream)
    i32 = lambda *sh_: torch.empty(*sh_, dtype=torch.int32, device=dev)
    f32 = lambda *sh_: torch.empty(*sh_, dtype=torch.float32, device=dev)
    out = AsymSciOutput(i32(B), i32(B, K + 1), f32(B, K + 1), f32(B, K + 1, 3), i32(B), i32(B, K + 1),
                        f32(B, K + 1), f32(B), i32(B))
    dt = _dtype_code(a)
    ws = workspace if workspace is not None else _workspace(dev, sh,
                                                            workspace_bytes(ASV_MODE_ASYMSPEC_SCI, B, K, V, dt))
    pc = _SciParamsC(params.T_base, params.alpha_omega, params.tau_credit, params.T_min, params.T_max,
                     params.ewma_beta)
    st = library().asymspec_sci_verify(_ptr(a), _ptr(b), _ptr(t), dt, _ptr(draft_ids), B, K, V, float(beta),
                                       float(gamma), C.byref(pc), _ptr(r_hat), _ptr(out.accept_len), _ptr(out.tokens),
                                       _ptr(out.D), _ptr(out.lse), _ptr(out.sci_accept_len), _ptr(out.sci_tokens),
                                       _ptr(out.jsd), _ptr(out.T), _ptr(out.req_status), _ptr(ws), ws.numel(), sh)
    _check(st, "asymspec_sci_verify")
    return out


def asymspec_verify_host(a, b, t, draft_ids, beta, gamma, arena: torch.Tensor, out_accept_len, out_tokens, out_D,
                         out_req_status, dtype: int, stream=None):
    """AsymSpec verification over host (pinned) buffers: raw addresses of CPU tensors; `arena`
    is a zeroed device uint8 tensor of host_arena_bytes() bytes.  Asynchronous on the stream."""
    if arena.get_device() != torch._C._cuda_getDevice():
        with torch.cuda.device(arena.device):
            return asymspec_verify_host(a, b, t, draft_ids, beta, gamma, arena, out_accept_len, out_tokens, out_D,
                                        out_req_status, dtype, stream)
    B, R1, V = a.shape
    K = R1 - 1
    sh = _stream_handle(arena.device, stream)
    st = library().asymspec_verify_host(_ptr(a), _ptr(b), _ptr(t), dtype, _ptr(draft_ids), B, K, V, float(beta),
                                        float(gamma), _ptr(out_accept_len), _ptr(out_tokens), _ptr(out_D),
                                        _ptr(out_req_status), _ptr(arena), arena.numel(), sh)
    _check(st, "asymspec_verify_host")


# ------------------------------------------------------------------ RAPID

@dataclass
class RapidOutput:
    accept_len: torch.Tensor
    tokens: torch.Tensor
    req_status: torch.Tensor


TAIL_KEEP_P = 0          # tail entries keep p, the head is rescaled (rapid_verify's reading)
TAIL_RENORMALISE_ALL = 1  # p substitutes phat on the tail, then every entry is renormalised


@_in_place
def rapid_verify(z: torch.Tensor, q: torch.Tensor, draft_ids: torch.Tensor, T: float = 1.0, eta: float = 10.0,
                 tail_frac: float = 0.1, seed: int = 1234, offset: int = 0, *, tail_mode: int = TAIL_KEEP_P,
                 out: Optional[RapidOutput] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> RapidOutput:
    """RAPID verification of fp32 target logits z and drafter probabilities q, [B, G+1, V]
    (`tail_mode` selects the reading of the tail protection, see rapid_verify_ex)."""
    _need_cuda(z, q, draft_ids)
    if z.dim() != 3 or z.shape != q.shape:
        raise AsvError(2, "z and q must share one [B, G+1, V] shape")
    if z.dtype != torch.float32 or q.dtype != torch.float32:
        raise AsvError(4, "RAPID takes float32 z and q")
    B, R1, V = z.shape
    G = R1 - 1
    if draft_ids.dtype != torch.int32 or tuple(draft_ids.shape) != (B, G):
        raise AsvError(2, "draft_ids must be int32 [B, G]")
    for n, x in (("z", z), ("q", q), ("draft_ids", draft_ids)):
        _contig(x, n)
    dev = z.device
    sh = _stream_handle(dev, stream)
    if out is None:
        out = RapidOutput(torch.empty(B, dtype=torch.int32, device=dev),
                          torch.empty(B, R1, dtype=torch.int32, device=dev),
                          torch.empty(B, dtype=torch.int32, device=dev))
    need = workspace_bytes(ASV_MODE_RAPID, B, G, V, ASV_F32)
    ws = workspace if workspace is not None else _workspace(dev, sh, need)
    opt = _RapidOptionsC(int(tail_mode))
    st = library().rapid_verify_ex(_ptr(z), _ptr(q), _ptr(draft_ids), B, G, V, float(T), float(eta),
                                   float(tail_frac), int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFF,
                                   C.byref(opt), _ptr(out.accept_len), _ptr(out.tokens), _ptr(out.req_status),
                                   _ptr(ws), ws.numel(), sh)
    _check(st, "rapid_verify_ex")
    return out


# ------------------------------------------------------------------ E2-SCI

@dataclass(frozen=True)
class SciParams:
    T_base: float = 0.3
    alpha_omega: float = 0.2
    tau_credit: float = 0.6
    T_min: float = 0.1
    T_max: float = 0.6
    ewma_beta: float = 0.3


@dataclass
class SciOutput:
    accept_len: torch.Tensor
    tokens: torch.Tensor
    jsd: torch.Tensor
    T: torch.Tensor
    req_status: torch.Tensor


@dataclass(frozen=True)
class SciStabilisers:
    """E2-SCI stabilisers (see sci_verify_ex in include/asv.h)."""
    hysteresis: float = 0.0
    min_refresh: int = 1
    fallback_acc: float = 0.0
    fallback_T: float = 0.1


def sci_state_new(B: int, device="cuda") -> torch.Tensor:
    """Zero-filled stabiliser state for B requests: [B, 4] int32 (16 bytes per request: T_applied
    as float64, then age and flags)."""
    return torch.zeros(B, 4, dtype=torch.int32, device=device)


def sci_state_decode(state: torch.Tensor):
    """(T_applied float64 [B], age int32 [B], flags int32 [B]) of a state tensor (copied to host)."""
    h = state.cpu().contiguous()
    return h[:, :2].contiguous().view(torch.float64).reshape(-1), h[:, 2].clone(), h[:, 3].clone()


@_in_place
def sci_verify(draft: torch.Tensor, target: torch.Tensor, draft_ids: torch.Tensor, r_hat: torch.Tensor,
               params: SciParams = SciParams(), *, stabilisers: Optional[SciStabilisers] = None,
               state: Optional[torch.Tensor] = None, prehit: bool = False, out: Optional[SciOutput] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> SciOutput:
    """One E2-SCI window; r_hat (float64 [B], device) is updated in place, and with `stabilisers`
    so is `state` (from sci_state_new).  `prehit` verifies every window's first draft first and
    drops windows whose first draft fails (sci_verify_prehit; no stabilisers)."""
    _need_cuda(draft, target, draft_ids, r_hat)
    if draft.dim() != 3 or draft.shape != target.shape or draft.dtype != target.dtype:
        raise AsvError(2, "draft and target must share one [B, K+1, V] shape and dtype")
    B, R1, V = draft.shape
    K = R1 - 1
    if draft_ids.dtype != torch.int32 or tuple(draft_ids.shape) != (B, K):
        raise AsvError(2, "draft_ids must be int32 [B, K]")
    if r_hat.dtype != torch.float64 or tuple(r_hat.shape) != (B,):
        raise AsvError(2, "r_hat must be float64 [B]")
    for n, x in (("draft", draft), ("target", target), ("draft_ids", draft_ids), ("r_hat", r_hat)):
        _contig(x, n)
    if stabilisers is not None:
        if state is None or state.dtype != torch.int32 or tuple(state.shape) != (B, 4) or not state.is_cuda:
            raise AsvError(2, "state must be an int32 [B, 4] CUDA tensor (sci_state_new)")
        _contig(state, "state")
    dev = draft.device
    sh = _stream_handle(dev, stream)
    if out is None:
        out = SciOutput(torch.empty(B, dtype=torch.int32, device=dev),
                        torch.empty(B, R1, dtype=torch.int32, device=dev),
                        torch.empty(B, R1, dtype=torch.float32, device=dev),
                        torch.empty(B, dtype=torch.float32, device=dev),
                        torch.empty(B, dtype=torch.int32, device=dev))
    dt = _dtype_code(draft)
    need = workspace_bytes(ASV_MODE_SCI, B, K, V, dt)
    ws = workspace if workspace is not None else _workspace(dev, sh, need)
    pc = _SciParamsC(params.T_base, params.alpha_omega, params.tau_credit, params.T_min, params.T_max,
                     params.ewma_beta)
    if prehit:
        if stabilisers is not None:
            raise AsvError(5, "the pre-hit path takes no stabilisers")
        st = library().sci_verify_prehit(_ptr(draft), _ptr(target), dt, _ptr(draft_ids), B, K, V, C.byref(pc),
                                         _ptr(r_hat), _ptr(out.accept_len), _ptr(out.tokens), _ptr(out.jsd),
                                         _ptr(out.T), _ptr(out.req_status), _ptr(ws), ws.numel(), sh)
        _check(st, "sci_verify_prehit")
        return out
    if stabilisers is None:
        st = library().sci_verify(_ptr(draft), _ptr(target), dt, _ptr(draft_ids), B, K, V, C.byref(pc), _ptr(r_hat),
                                  _ptr(out.accept_len), _ptr(out.tokens), _ptr(out.jsd), _ptr(out.T),
                                  _ptr(out.req_status), _ptr(ws), ws.numel(), sh)
        _check(st, "sci_verify")
        return out
    sc = _SciStabC(float(stabilisers.hysteresis), int(stabilisers.min_refresh), 0, float(stabilisers.fallback_acc),
                   float(stabilisers.fallback_T))
    st = library().sci_verify_ex(_ptr(draft), _ptr(target), dt, _ptr(draft_ids), B, K, V, C.byref(pc), C.byref(sc),
                                 _ptr(r_hat), _ptr(state), _ptr(out.accept_len), _ptr(out.tokens), _ptr(out.jsd),
                                 _ptr(out.T), _ptr(out.req_status), _ptr(ws), ws.numel(), sh)
    _check(st, "sci_verify_ex")
    return out


# ------------------------------------------------------------------ paged key/value cache

@dataclass
class PagedAppendOutput:
    q: Optional[torch.Tensor]  # [N, q_heads, head_dim] rotated queries (None without q)
    req_status: torch.Tensor   # [B] int32 (ASV_REQ_* bits, ORed in)


@dataclass
class PagedAttentionOutput:
    out: torch.Tensor            # [N, q_heads, head_dim]
    lse: Optional[torch.Tensor]  # [N, q_heads] float32 (natural log; may be None)
    req_status: torch.Tensor     # [B] int32 (ASV_REQ_* bits, ORed in)


_ext = None


def _paged_ext():
    """The binding's compiled module, bound to the library's paged entry points."""
    global _ext
    L = library()
    with _lib_lock:
        if _ext is None:
            if not os.path.exists(_build.TORCH_EXT):
                raise AsvError(-1, f"asv_torch.so not built ({_build.TORCH_EXT}); call speculative_decoding_logit_gb300.build()")
            if not _build.torch_ext_fits():
                raise AsvError(-1, f"{_build.TORCH_EXT} was built for another PyTorch; call speculative_decoding_logit_gb300.build()")
            loader = importlib.machinery.ExtensionFileLoader("asv_torch", _build.TORCH_EXT)
            ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("asv_torch", loader))
            loader.exec_module(ext)
            ext.bind(AsvError, *(C.cast(f, C.c_void_p).value for f in (L.paged_attention, L.paged_kv_append,
                                                                        L.asv_status_string, L.asv_last_cuda_error)))
            _ext = ext
    return _ext


def _raw_stream(t: torch.Tensor, stream) -> Optional[int]:
    """The CUDA stream handle of `stream`, or of the current stream of t's device; None where that device is not the
    current one (a launch goes to the current device)."""
    dev = t.get_device()
    if dev < 0:
        _need_cuda(t)
    if stream is not None and stream.device != t.device:
        raise AsvError(2, "the stream must be one of the tensors' device")
    if dev != torch._C._cuda_getDevice():
        return None
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def paged_kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_table: torch.Tensor, cache_len: torch.Tensor, indptr: torch.Tensor, *,
                    q: Optional[torch.Tensor] = None, rotary: Optional[torch.Tensor] = None,
                    interleaved: bool = False, out: Optional[PagedAppendOutput] = None,
                    stream=None) -> PagedAppendOutput:
    """Appends the packed new tokens' keys and values ([N, kv_heads, head_dim]; request b's are rows
    indptr[b]..indptr[b+1]) to the paged caches at positions cache_len[b] onwards; with `rotary`
    ([max_position, dim] float32: cos of the dim/2 angles of each position, then their sines) the keys
    are rotated on the way, and the queries `q` into out.q, which must not overlap them (paged_kv_append in
    include/asv.h).  cache_len is not advanced.  The caches take any positive strides that are multiples of 8 elements,
    head rows contiguous.  With `stream`, the call's order with other streams' work is the caller's business; what it
    makes for `out` belongs to that stream."""
    handle = _raw_stream(k, stream)
    if handle is None:
        with torch.cuda.device(k.device):
            return paged_kv_append(k, v, k_cache, v_cache, block_table, cache_len, indptr, q=q, rotary=rotary,
                                   interleaved=interleaved, out=out, stream=stream)
    if out is None:
        dev = k.device
        out = PagedAppendOutput(*_made_on(stream, lambda: (
            None if q is None else torch.empty(q.shape, dtype=q.dtype, device=dev),
            torch.zeros(cache_len.shape, dtype=torch.int32, device=dev))))
    (_ext or _paged_ext()).paged_kv_append(k, v, k_cache, v_cache, block_table, cache_len, indptr, q, rotary,
                                           interleaved, out.q, out.req_status, handle)
    return out


# Workspaces of paged_attention, one per (device, stream): their partial results are not zeroed by a
# call, so they are kept apart from the verification's.  Only their first bytes have to start at zero.
_paged_ws_cache: dict = {}
PAGED_WORKSPACE_ZEROED = 4096


def clear_workspaces():
    """Zero-fills the workspaces that calls without workspace= keep for each stream, in place, when everything queued on
    their devices is done.  To be called after a request came back with REQ_TIMEOUT: the call that gave up may have
    left its workspace dirty, which later calls would count on."""
    with _ws_lock:
        kept = list(_ws_cache.values()) + [ws[:PAGED_WORKSPACE_ZEROED] for ws in _paged_ws_cache.values()]
        devices = {ws.device for ws in kept}
        for d in devices:
            torch.cuda.synchronize(d)
        for ws in kept:
            ws.zero_()
        for d in devices:
            torch.cuda.synchronize(d)


def paged_workspace_bytes(q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace one paged_attention call with these heads needs, for any batch."""
    return int(library().asv_paged_workspace_bytes(q_heads, kv_heads, head_dim))


def _paged_workspace(q: torch.Tensor, handle: int, stream) -> torch.Tensor:
    """A new workspace for any heads, kept for the stream's later calls unless it is capturing (what is
    allocated then belongs to the graph, and is zeroed by its replays only)."""
    with _ws_lock, torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(q.device)):
        ws = torch.empty(paged_workspace_bytes(1, 1, 128), dtype=torch.uint8, device=q.device)
        ws[:PAGED_WORKSPACE_ZEROED].zero_()
        if not torch.cuda.is_current_stream_capturing():
            _paged_ws_cache[q.get_device(), handle] = ws
    return ws


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    cache_len: torch.Tensor, indptr: torch.Tensor, *, scale: Optional[float] = None,
                    window: int = 0, out: Optional[PagedAttentionOutput] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> PagedAttentionOutput:
    """Attention of the packed chunks of new tokens q [N, q_heads, head_dim] over the paged caches, the
    chunk's own tokens (appended before, see paged_kv_append) included: causal, grouped heads, with
    `window` > 0 only the last `window` positions of each token (paged_attention in include/asv.h).
    cache_len [B] counts the tokens before the chunk; scale defaults to head_dim ** -0.5.  `stream` as for
    paged_kv_append.  Without `workspace` the call uses one kept for its stream (40 MB), and so does a graph captured
    there: give a workspace of its own (paged_workspace_bytes, its first PAGED_WORKSPACE_ZEROED bytes zero) to a graph
    that may be replayed next to the stream's other calls."""
    handle = _raw_stream(q, stream)
    if handle is None:
        with torch.cuda.device(q.device):
            return paged_attention(q, k_cache, v_cache, block_table, cache_len, indptr, scale=scale, window=window,
                                   out=out, workspace=workspace, stream=stream)
    if out is None:
        dev = q.device
        out = PagedAttentionOutput(*_made_on(stream, lambda: (
            torch.empty(q.shape, dtype=q.dtype, device=dev),
            torch.empty(q.shape[:2], dtype=torch.float32, device=dev),
            torch.zeros(cache_len.shape, dtype=torch.int32, device=dev))))
    if workspace is None:
        workspace = _paged_ws_cache.get((q.get_device(), handle))
        if workspace is None:
            workspace = _paged_workspace(q, handle, stream)
    (_ext or _paged_ext()).paged_attention(q, k_cache, v_cache, block_table, cache_len, indptr, scale, window,
                                           out.out, out.lse, out.req_status, workspace, handle)
    return out
