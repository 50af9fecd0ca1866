"""Thin ctypes binding of libssd's C ABI (include/ssd.h).

Argument marshalling only: shapes, dtypes, devices and contiguity of torch
tensors are checked, then raw device pointers and the current HIP stream are
handed to the library.  Every step of the scan runs in the library's HIP
kernels; there is no fallback of any kind.  torch only provides device memory
(including the workspace) and the stream.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssd.so")

SSD_OK = 0
STATUS_NAMES = {0: "SSD_OK", 1: "SSD_ERR_NULL_ARG", 2: "SSD_ERR_BAD_SHAPE", 3: "SSD_ERR_UNSUPPORTED",
                4: "SSD_ERR_WORKSPACE", 5: "SSD_ERR_BAD_INPUT", 6: "SSD_ERR_HIP", 7: "SSD_ERR_MISALIGNED",
                8: "SSD_ERR_SCRATCH"}

# every symbol include/ssd.h declares
EXPORTED = ("ssd_abi_version", "ssd_status_string", "ssd_workspace_size",
            "ssd_workspace_get_layout", "ssd_chunk_scan_varlen_fwd_inplace",
            "ssd_kernel_count", "ssd_kernel_name", "ssd_chunk_scan_varlen_fwd_inplace_profiled",
            "ssd_chunk_scan_varlen_fwd", "ssd_chunk_scan_varlen_fwd_profiled", "ssd_validate_inputs",
            "ssd_chunk_scan_varlen_fwd_inplace_noalloc",
            "ssd_linear_attn_workspace_size", "ssd_linear_attn_varlen_fwd_inplace", "ssd_linear_attn_varlen_fwd",
            "ssd_linear_attn_varlen_bwd", "ssd_linear_attn_step_inplace", "ssd_state_quantize",
            "ssd_state_dequantize",
            "ssd_rms_norm_fwd", "ssd_rms_norm_workspace_size", "ssd_rms_norm_bwd",
            "ssd_causal_conv_varlen_fwd_inplace", "ssd_causal_conv_varlen_fwd", "ssd_causal_conv_workspace_size",
            "ssd_causal_conv_varlen_bwd", "ssd_causal_conv_step_inplace",
            "ssd_selective_scan_workspace_size", "ssd_selective_scan_varlen_fwd_inplace",
            "ssd_selective_scan_varlen_fwd", "ssd_selective_scan_varlen_bwd", "ssd_selective_scan_step_inplace")


class SsdError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class ssd_problem(ctypes.Structure):
    _fields_ = [("total_len", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("nheads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("ngroups", ctypes.c_int32), ("dstate", ctypes.c_int32),
                ("max_slots", ctypes.c_int32), ("chunk_size", ctypes.c_int32),
                ("dt_softplus", ctypes.c_int32), ("state_dtype", ctypes.c_int32),
                ("short_path_max", ctypes.c_int32)]


class ssd_linear_attn_problem(ctypes.Structure):
    _fields_ = [("total_len", ctypes.c_int64), ("batch", ctypes.c_int32), ("nheads", ctypes.c_int32),
                ("ngroups", ctypes.c_int32), ("key_dim", ctypes.c_int32), ("value_dim", ctypes.c_int32),
                ("max_slots", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64)]


class ssd_state_cache_problem(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("nheads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dstate", ctypes.c_int32), ("max_slots", ctypes.c_int32), ("max_entries", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32), ("code_format", ctypes.c_int32)]


class ssd_norm_problem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int32), ("residual_dtype", ctypes.c_int32),
                ("out_format", ctypes.c_int32), ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64)]


class ssd_conv_problem(ctypes.Structure):
    _fields_ = [("total_len", ctypes.c_int64), ("batch", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("width", ctypes.c_int32), ("max_slots", ctypes.c_int32), ("silu", ctypes.c_int32),
                ("x_stride", ctypes.c_int64)]


class ssd_selective_problem(ctypes.Structure):
    _fields_ = [("total_len", ctypes.c_int64), ("batch", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("ngroups", ctypes.c_int32), ("dstate", ctypes.c_int32), ("max_slots", ctypes.c_int32),
                ("dt_softplus", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("dt_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64), ("b_stride", ctypes.c_int64),
                ("c_stride", ctypes.c_int64)]


class ssd_workspace_layout(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_size_t), ("nchunks_max", ctypes.c_int64),
                ("meta", ctypes.c_size_t), ("chunk_off", ctypes.c_size_t),
                ("desc", ctypes.c_size_t), ("dts", ctypes.c_size_t), ("cs2", ctypes.c_size_t),
                ("cbt", ctypes.c_size_t), ("gexp", ctypes.c_size_t),
                ("states", ctypes.c_size_t), ("sexp", ctypes.c_size_t),
                ("hin", ctypes.c_size_t), ("hexp", ctypes.c_size_t), ("xexp", ctypes.c_size_t),
                ("seq_list", ctypes.c_size_t), ("recur_list", ctypes.c_size_t),
                ("core_nheads", ctypes.c_int32), ("core_dstate", ctypes.c_int32),
                ("x_pad", ctypes.c_size_t), ("y_pad", ctypes.c_size_t), ("bc_pad", ctypes.c_size_t),
                ("head_wide", ctypes.c_size_t), ("state_pad", ctypes.c_size_t)]


_lock = threading.Lock()
_lib = None

# SSD_ABI_VERSION of include/ssd.h that the ctypes structures below mirror
ABI_VERSION = 18
NOALLOC_SCRATCH_BYTES = 64 << 20  # SSD_NOALLOC_SCRATCH_BYTES
STATE_F32, STATE_BF16 = 0, 1  # SSD_STATE_F32, SSD_STATE_BF16
SHORT_PATH_LIMIT = 128  # SSD_SHORT_PATH_LIMIT
MAX_DSTATE, MAX_HEAD_DIM = 256, 1024  # SSD_MAX_DSTATE, SSD_MAX_HEAD_DIM
LINEAR_ATTN_MAX_DIM = 256  # SSD_LINEAR_ATTN_MAX_DIM
CODE_I8, CODE_E4M3 = 0, 1  # SSD_CODE_I8, SSD_CODE_E4M3
OUT_BF16 = 2  # SSD_OUT_BF16
NORM_MAX_WIDTH = 32768  # SSD_NORM_MAX_WIDTH
CONV_MAX_WIDTH = 4  # SSD_CONV_MAX_WIDTH
SELECTIVE_MAX_DSTATE = 64  # SSD_SELECTIVE_MAX_DSTATE
SHORT_PATH_DEFAULT = -1  # ssd_problem.short_path_max: any negative value selects SHORT_PATH_LIMIT


def load_library():
    """Load libssd.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it first "
                    "(python -m mamba_ssd_chunked_chunk_amd.build)")
            lib = ctypes.CDLL(LIB_PATH)
            V = ctypes.c_void_p
            PP = ctypes.POINTER(ssd_problem)
            lib.ssd_abi_version.restype = ctypes.c_int
            lib.ssd_abi_version.argtypes = []
            if lib.ssd_abi_version() != ABI_VERSION:
                raise RuntimeError(f"{LIB_PATH} has ABI version {lib.ssd_abi_version()}, the binding "
                                   f"expects {ABI_VERSION}: rebuild it")
            lacks = [name for name in EXPORTED if not hasattr(lib, name)]
            if lacks:
                raise RuntimeError(f"{LIB_PATH} lacks {', '.join(lacks)}: rebuild it")
            lib.ssd_status_string.restype = ctypes.c_char_p
            lib.ssd_status_string.argtypes = [ctypes.c_int]
            lib.ssd_workspace_size.restype = ctypes.c_int
            lib.ssd_workspace_size.argtypes = [PP, ctypes.POINTER(ctypes.c_size_t)]
            lib.ssd_workspace_get_layout.restype = ctypes.c_int
            lib.ssd_workspace_get_layout.argtypes = [PP, ctypes.POINTER(ssd_workspace_layout)]
            lib.ssd_chunk_scan_varlen_fwd_inplace.restype = ctypes.c_int
            lib.ssd_chunk_scan_varlen_fwd_inplace.argtypes = [PP] + [V] * 13 + [ctypes.c_size_t, V]
            lib.ssd_kernel_count.restype = ctypes.c_int
            lib.ssd_kernel_count.argtypes = []
            lib.ssd_kernel_name.restype = ctypes.c_char_p
            lib.ssd_kernel_name.argtypes = [ctypes.c_int]
            lib.ssd_chunk_scan_varlen_fwd_inplace_profiled.restype = ctypes.c_int
            lib.ssd_chunk_scan_varlen_fwd_inplace_profiled.argtypes = (
                [PP] + [V] * 13 + [ctypes.c_size_t, V, ctypes.POINTER(ctypes.c_void_p), ctypes.c_int])
            lib.ssd_chunk_scan_varlen_fwd.restype = ctypes.c_int
            lib.ssd_chunk_scan_varlen_fwd.argtypes = [PP] + [V] * 12 + [ctypes.c_size_t, V]
            lib.ssd_chunk_scan_varlen_fwd_profiled.restype = ctypes.c_int
            lib.ssd_chunk_scan_varlen_fwd_profiled.argtypes = (
                [PP] + [V] * 12 + [ctypes.c_size_t, V, ctypes.POINTER(ctypes.c_void_p), ctypes.c_int])
            lib.ssd_chunk_scan_varlen_fwd_inplace_noalloc.restype = ctypes.c_int
            lib.ssd_chunk_scan_varlen_fwd_inplace_noalloc.argtypes = [PP] + [V] * 12 + [V]
            lib.ssd_validate_inputs.restype = ctypes.c_int
            lib.ssd_validate_inputs.argtypes = [PP, V, V, V]
            PL = ctypes.POINTER(ssd_linear_attn_problem)
            PC = ctypes.POINTER(ssd_state_cache_problem)
            PN, PV, PS = (ctypes.POINTER(s) for s in (ssd_norm_problem, ssd_conv_problem, ssd_selective_problem))
            for name, args in (
                    ("ssd_linear_attn_workspace_size", [PL, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]),
                    ("ssd_linear_attn_varlen_fwd_inplace", [PL] + [V] * 10 + [ctypes.c_size_t, V]),
                    ("ssd_linear_attn_varlen_fwd", [PL] + [V] * 9 + [ctypes.c_size_t, V]),
                    ("ssd_linear_attn_varlen_bwd", [PL] + [V] * 13 + [ctypes.c_size_t, V]),
                    ("ssd_linear_attn_step_inplace", [PL] + [V] * 9),
                    ("ssd_state_quantize", [PC] + [V] * 6),
                    ("ssd_state_dequantize", [PC] + [V] * 6),
                    ("ssd_rms_norm_fwd", [PN] + [V] * 7),
                    ("ssd_rms_norm_workspace_size", [PN, ctypes.POINTER(ctypes.c_size_t)]),
                    ("ssd_rms_norm_bwd", [PN] + [V] * 8 + [ctypes.c_size_t, V]),
                    ("ssd_causal_conv_varlen_fwd_inplace", [PV] + [V] * 9),
                    ("ssd_causal_conv_varlen_fwd", [PV] + [V] * 8),
                    ("ssd_causal_conv_workspace_size", [PV, ctypes.POINTER(ctypes.c_size_t)]),
                    ("ssd_causal_conv_varlen_bwd", [PV] + [V] * 12 + [ctypes.c_size_t, V]),
                    ("ssd_causal_conv_step_inplace", [PV] + [V] * 8),
                    ("ssd_selective_scan_workspace_size", [PS, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]),
                    ("ssd_selective_scan_varlen_fwd_inplace", [PS] + [V] * 14 + [ctypes.c_size_t, V]),
                    ("ssd_selective_scan_varlen_fwd", [PS] + [V] * 13 + [ctypes.c_size_t, V]),
                    ("ssd_selective_scan_varlen_bwd", [PS] + [V] * 22 + [ctypes.c_size_t, V]),
                    ("ssd_selective_scan_step_inplace", [PS] + [V] * 13)):
                getattr(lib, name).restype = ctypes.c_int
                getattr(lib, name).argtypes = args
            _lib = lib
    return _lib


def _check(status: int, what: str):
    if status != SSD_OK:
        lib = load_library()
        msg = lib.ssd_status_string(status).decode()
        raise SsdError(status, f"{what}: {msg}")


def make_problem(total_len, batch, nheads, head_dim, ngroups, dstate, max_slots,
                 dt_softplus=True, chunk_size=0, state_dtype=STATE_F32,
                 short_path_max=SHORT_PATH_DEFAULT) -> ssd_problem:
    return ssd_problem(int(total_len), int(batch), int(nheads), int(head_dim), int(ngroups),
                       int(dstate), int(max_slots), int(chunk_size), 1 if dt_softplus else 0,
                       int(state_dtype), int(short_path_max))


def _state_dtype(t, name):
    """SSD_STATE_* of a state tensor (fp32 or bf16)."""
    import torch
    if t.dtype == torch.float32:
        return STATE_F32
    if t.dtype == torch.bfloat16:
        return STATE_BF16
    raise TypeError(f"{name}: expected float32 or bfloat16 states, got {t.dtype}")


def ssd_abi_version() -> int:
    return load_library().ssd_abi_version()


def ssd_workspace_size(prob: ssd_problem) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_workspace_size(ctypes.byref(prob), ctypes.byref(n)), "ssd_workspace_size")
    return n.value


def ssd_workspace_get_layout(prob: ssd_problem) -> dict:
    L = ssd_workspace_layout()
    _check(load_library().ssd_workspace_get_layout(ctypes.byref(prob), ctypes.byref(L)),
           "ssd_workspace_get_layout")
    return {name: getattr(L, name) for name, _ in ssd_workspace_layout._fields_}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, dtype, shape, device):
    import torch
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return torch


def _opt(t, name, dtype, shape, device):
    if t is None or t.numel() == 0:
        return None
    _need(t, name, dtype, shape, device)
    return t


def _need_workspace(t, need, device):
    """A workspace has to hold its bytes itself (an expanded byte has their number, not their memory)."""
    import torch
    if t.dtype != torch.uint8 or t.numel() < need or t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor of >= {need} bytes on {device}")


def problem_from_tensors(x, B, ssm_pool, query_start_loc, dt_softplus=True,
                         short_path_max=SHORT_PATH_DEFAULT) -> ssd_problem:
    T, H, P = x.shape
    _, G, N = B.shape
    return make_problem(T, query_start_loc.numel() - 1, H, P, G, N, ssm_pool.shape[0], dt_softplus,
                        state_dtype=_state_dtype(ssm_pool, "ssm_pool"), short_path_max=short_path_max)


def ssd_chunk_scan_varlen_fwd_inplace(y, x, dt, A, B, C, D, dt_bias, ssm_pool, query_start_loc,
                                      has_initial_state, cache_indices, *, dt_softplus=True,
                                      short_path_max=SHORT_PATH_DEFAULT, workspace=None, stream=None):
    """In-place varlen SSD forward (see include/ssd.h for the semantics).

    Tensors (torch, on one HIP device, contiguous): y, x bf16 [T,H,P];
    dt fp32 [T,H]; A fp32 [H]; B, C bf16 [T,G,N]; D, dt_bias fp32 [H] or
    None/empty; ssm_pool fp32 [S,H,P,N] (updated in place);
    query_start_loc int32 [batch+1]; has_initial_state uint8/bool [batch] or
    None/empty; cache_indices int32/uint32 [batch] (reinterpreted as uint32).
    ``workspace``: uint8 tensor of at least ssd_workspace_size() bytes, or
    None to allocate one.  Runs on ``stream`` (a torch.cuda.Stream) or the
    current stream; asynchronous.  Returns the workspace tensor.  A bf16
    ssm_pool selects bf16 state storage (arithmetic stays fp32).
    ``short_path_max``: longest sequence the short path takes (dstate <= 128;
    0: none, negative: the library default SHORT_PATH_LIMIT).
    """
    import torch
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssd runs on a HIP device; got tensors on " + str(dev))
    T, H, P = x.shape
    if B.dim() != 3:
        raise ValueError("B must be [T, G, N]")
    G, N = B.shape[1], B.shape[2]
    batch = query_start_loc.numel() - 1
    S = ssm_pool.shape[0]
    _need(y, "y", torch.bfloat16, (T, H, P), dev)
    _need(x, "x", torch.bfloat16, (T, H, P), dev)
    _need(dt, "dt", torch.float32, (T, H), dev)
    _need(A, "A", torch.float32, (H,), dev)
    _need(B, "B", torch.bfloat16, (T, G, N), dev)
    _need(C, "C", torch.bfloat16, (T, G, N), dev)
    D = _opt(D, "D", torch.float32, (H,), dev)
    dt_bias = _opt(dt_bias, "dt_bias", torch.float32, (H,), dev)
    sd = _state_dtype(ssm_pool, "ssm_pool")
    _need(ssm_pool, "ssm_pool", ssm_pool.dtype, (S, H, P, N), dev)
    _need(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    if has_initial_state is not None and has_initial_state.numel() > 0:
        if has_initial_state.dtype == torch.bool:
            has_initial_state = has_initial_state.view(torch.uint8)
        _need(has_initial_state, "has_initial_state", torch.uint8, (batch,), dev)
    else:
        has_initial_state = None
    if cache_indices.dtype not in (torch.int32, torch.uint32):
        raise TypeError("cache_indices must be int32 or uint32")
    if tuple(cache_indices.shape) != (batch,) or not cache_indices.is_contiguous() or cache_indices.device != dev:
        raise ValueError("cache_indices must be a contiguous [batch] tensor on the same device")
    prob = make_problem(T, batch, H, P, G, N, S, dt_softplus, state_dtype=sd, short_path_max=short_path_max)
    need = ssd_workspace_size(prob)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need_workspace(workspace, need, dev)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    status = load_library().ssd_chunk_scan_varlen_fwd_inplace(
        ctypes.byref(prob), _ptr(y), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(dt_bias), _ptr(ssm_pool), _ptr(query_start_loc), _ptr(has_initial_state),
        _ptr(cache_indices), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
        ctypes.c_void_p(st.cuda_stream))
    _check(status, "ssd_chunk_scan_varlen_fwd_inplace")
    return workspace


def ssd_chunk_scan_varlen_fwd_inplace_noalloc(y, x, dt, A, B, C, D, dt_bias, ssm_pool, query_start_loc,
                                              has_initial_state, cache_indices, *, dt_softplus=True,
                                              short_path_max=SHORT_PATH_DEFAULT, stream=None):
    """The in-place operation without a workspace argument: the library's
    own scratch array (NOALLOC_SCRATCH_BYTES per GPU) holds the
    intermediates, and nothing is allocated.  Same tensors and checks as
    ssd_chunk_scan_varlen_fwd_inplace; calls that can overlap on one GPU race
    on the shared scratch (one stream orders them)."""
    import torch
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssd runs on a HIP device; got tensors on " + str(dev))
    T, H, P = x.shape
    if B.dim() != 3:
        raise ValueError("B must be [T, G, N]")
    G, N = B.shape[1], B.shape[2]
    batch = query_start_loc.numel() - 1
    S = ssm_pool.shape[0]
    _need(y, "y", torch.bfloat16, (T, H, P), dev)
    _need(x, "x", torch.bfloat16, (T, H, P), dev)
    _need(dt, "dt", torch.float32, (T, H), dev)
    _need(A, "A", torch.float32, (H,), dev)
    _need(B, "B", torch.bfloat16, (T, G, N), dev)
    _need(C, "C", torch.bfloat16, (T, G, N), dev)
    D = _opt(D, "D", torch.float32, (H,), dev)
    dt_bias = _opt(dt_bias, "dt_bias", torch.float32, (H,), dev)
    sd = _state_dtype(ssm_pool, "ssm_pool")
    _need(ssm_pool, "ssm_pool", ssm_pool.dtype, (S, H, P, N), dev)
    _need(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    if has_initial_state is not None and has_initial_state.numel() > 0:
        if has_initial_state.dtype == torch.bool:
            has_initial_state = has_initial_state.view(torch.uint8)
        _need(has_initial_state, "has_initial_state", torch.uint8, (batch,), dev)
    else:
        has_initial_state = None
    if cache_indices.dtype not in (torch.int32, torch.uint32):
        raise TypeError("cache_indices must be int32 or uint32")
    if tuple(cache_indices.shape) != (batch,) or not cache_indices.is_contiguous() or cache_indices.device != dev:
        raise ValueError("cache_indices must be a contiguous [batch] tensor on the same device")
    prob = make_problem(T, batch, H, P, G, N, S, dt_softplus, state_dtype=sd, short_path_max=short_path_max)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    status = load_library().ssd_chunk_scan_varlen_fwd_inplace_noalloc(
        ctypes.byref(prob), _ptr(y), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(dt_bias), _ptr(ssm_pool), _ptr(query_start_loc), _ptr(has_initial_state),
        _ptr(cache_indices), ctypes.c_void_p(st.cuda_stream))
    _check(status, "ssd_chunk_scan_varlen_fwd_inplace_noalloc")


def ssd_chunk_scan_varlen_fwd(y, x, dt, A, B, C, D, dt_bias, initial_states, final_states,
                              query_start_loc, *, dt_softplus=True, short_path_max=SHORT_PATH_DEFAULT,
                              workspace=None, stream=None):
    """Varlen SSD forward with separate initial and final states (see
    include/ssd.h): sequence b starts from ``initial_states[b]`` ([batch,H,P,N],
    or None/empty for zero) and its final state is written to
    ``final_states[b]`` ([batch,H,P,N]); both fp32, or both bf16 (bf16 state
    storage, arithmetic in fp32).  Other tensors as for
    ssd_chunk_scan_varlen_fwd_inplace.  Returns the workspace tensor.
    """
    import torch
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssd runs on a HIP device; got tensors on " + str(dev))
    T, H, P = x.shape
    if B.dim() != 3:
        raise ValueError("B must be [T, G, N]")
    G, N = B.shape[1], B.shape[2]
    batch = query_start_loc.numel() - 1
    _need(y, "y", torch.bfloat16, (T, H, P), dev)
    _need(x, "x", torch.bfloat16, (T, H, P), dev)
    _need(dt, "dt", torch.float32, (T, H), dev)
    _need(A, "A", torch.float32, (H,), dev)
    _need(B, "B", torch.bfloat16, (T, G, N), dev)
    _need(C, "C", torch.bfloat16, (T, G, N), dev)
    D = _opt(D, "D", torch.float32, (H,), dev)
    dt_bias = _opt(dt_bias, "dt_bias", torch.float32, (H,), dev)
    if final_states is None:
        raise ValueError("final_states is required")
    sd = _state_dtype(final_states, "final_states")
    initial_states = _opt(initial_states, "initial_states", final_states.dtype, (batch, H, P, N), dev)
    _need(final_states, "final_states", final_states.dtype, (batch, H, P, N), dev)
    _need(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    prob = make_problem(T, batch, H, P, G, N, max(batch, 1), dt_softplus, state_dtype=sd,
                        short_path_max=short_path_max)
    need = ssd_workspace_size(prob)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need_workspace(workspace, need, dev)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    status = load_library().ssd_chunk_scan_varlen_fwd(
        ctypes.byref(prob), _ptr(y), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(dt_bias), _ptr(initial_states), _ptr(final_states), _ptr(query_start_loc),
        _ptr(workspace), ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(st.cuda_stream))
    _check(status, "ssd_chunk_scan_varlen_fwd")
    return workspace


def ssd_validate_inputs(prob: ssd_problem, query_start_loc, cache_indices, stream=None) -> int:
    """Synchronous precondition check; returns the status code."""
    import torch
    st = stream if stream is not None else torch.cuda.current_stream(query_start_loc.device)
    return load_library().ssd_validate_inputs(ctypes.byref(prob), _ptr(query_start_loc),
                                              _ptr(cache_indices), ctypes.c_void_p(st.cuda_stream))


# ---------------------------------------------------------------------------
# linear attention with a fixed decay per head, and the 8-bit state cache.
# Decode steps call these once a layer and token, so what they check they check
# in few operations: _inputs() imports torch once, addresses go to ctypes as
# they are, and problems are made once for each set of sizes.

torch = None  # imported by the first call


def _raw_stream(dev):
    """Handle of the device's current stream."""
    return torch.cuda.current_stream(dev).cuda_stream


def _import_torch():
    global torch, _raw_stream
    import torch as module
    torch = module
    handle = getattr(module._C, "_cuda_getCurrentRawStream", None)
    if handle is not None:  # the same without a Stream object
        _raw_stream = lambda dev: handle(dev.index)  # noqa: E731


def make_linear_attn_problem(total_len, batch, nheads, ngroups, key_dim, value_dim, max_slots=1,
                             state_dtype=STATE_F32, scale=1.0, q_stride=0, k_stride=0,
                             v_stride=0) -> ssd_linear_attn_problem:
    return ssd_linear_attn_problem(int(total_len), int(batch), int(nheads), int(ngroups), int(key_dim),
                                   int(value_dim), int(max_slots), int(state_dtype), float(scale), int(q_stride),
                                   int(k_stride), int(v_stride))


def ssd_linear_attn_workspace_size(prob: ssd_linear_attn_problem, backward=False) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_linear_attn_workspace_size(ctypes.byref(prob), 1 if backward else 0, ctypes.byref(n)),
           "ssd_linear_attn_workspace_size")
    return n.value


def _refuse_tensor(t, name, dtype, shape, device):
    """Why a tensor is not a dense one of this type and shape on the device."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


def _dense(t, name, dtype, shape, device):
    """Address of a dense tensor of this type and shape on the device (one test where all is well)."""
    if t is None or t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _refuse_tensor(t, name, dtype, shape, device)
    return t.data_ptr()


def _dense_or_none(t, name, dtype, shape, device):
    return None if t is None or t.numel() == 0 else _dense(t, name, dtype, shape, device)


def _token_stride(t, name, shape, device):
    """Elements between tokens of a bf16 [T, n, D] tensor whose tokens are dense rows (a slice of a wider
    projection is one); 0 for a dense tensor."""
    if torch is None:
        _import_torch()
    if t.dtype != torch.bfloat16 or t.shape != shape or t.device != device:
        _refuse_tensor(t, name, torch.bfloat16, shape, device)
    if t.is_contiguous():
        return 0
    T, n, D = shape
    if (D > 1 and t.stride(2) != 1) or (n > 1 and t.stride(1) != D):
        raise ValueError(f"{name}: the heads of a token must be dense")
    if T > 1 and (t.stride(0) < n * D or t.stride(0) % 8 != 0):
        raise ValueError(f"{name}: the stride between tokens must be a multiple of 8 elements, at least {n * D}")
    return t.stride(0) if T > 1 else 0


@functools.lru_cache(maxsize=256)
def _linear_attn_sizes(backward, *sizes):
    """(reference to the problem of these sizes, workspace bytes); ``backward`` None: of single tokens, which need
    none and have wider limits"""
    prob = make_linear_attn_problem(*sizes)
    return ctypes.byref(prob), 0 if backward is None else ssd_linear_attn_workspace_size(prob, backward)


def _linear_attn(q, k, v, log_decay, batch, max_slots, state_dtype, scale, backward):
    """What a linear-attention call goes by, its inputs checked: problem and workspace bytes (of the direction, or
    None for single tokens), device, shape of a state, addresses of q, k, v and log_decay."""
    if torch is None:
        _import_torch()
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t is None or t.dim() != 3:
            raise ValueError(f"{name} must be [T, heads, dim]")
    dev = v.device
    if dev.type != "cuda":
        raise ValueError("libssd runs on a HIP device; got tensors on " + str(dev))
    T, H, V = v.shape
    _, G, K = qk = q.shape
    if qk[0] != T:
        _refuse_tensor(q, "q", torch.bfloat16, (T, G, K), dev)
    prob, need = _linear_attn_sizes(
        backward, T, batch, H, G, K, V, max_slots, state_dtype, K ** -0.5 if scale is None else float(scale),
        _token_stride(q, "q", qk, dev), _token_stride(k, "k", qk, dev), _token_stride(v, "v", (T, H, V), dev))
    decay = _dense(log_decay, "log_decay", torch.float32, (H,), dev)
    return prob, need, dev, (H, V, K), (q.data_ptr(), k.data_ptr(), v.data_ptr(), decay)


def _slots(cache_indices, has_initial_state, batch, dev):
    """Addresses of cache_indices and has_initial_state (or None), checked."""
    if cache_indices.dtype not in (torch.int32, torch.uint32):
        raise TypeError("cache_indices must be int32 or uint32")
    idx = _dense(cache_indices, "cache_indices", cache_indices.dtype, (batch,), dev)
    if has_initial_state is None or has_initial_state.numel() == 0:
        return idx, None
    if has_initial_state.dtype == torch.bool:
        has_initial_state = has_initial_state.view(torch.uint8)
    return idx, _dense(has_initial_state, "has_initial_state", torch.uint8, (batch,), dev)


def _launch(name, dev, stream, call):
    """Runs ``call(stream)`` on the stream (the current one for None) with the tensors' device current, and raises
    what it returns."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    if dev.index == torch.cuda.current_device():
        status = call(_raw_stream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            status = call(_raw_stream(dev) if stream is None else stream.cuda_stream)
    if status != SSD_OK:
        _check(status, name)


def _run(name, dev, stream, need, workspace, call):
    """The same for ``call(workspace address, bytes, stream)``.  A workspace that the caller does not give is
    allocated on the call's stream.  Returns the workspace (None where none was given and none is needed)."""
    if workspace is not None:
        _need_workspace(workspace, need, dev)
    elif need:
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    at, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _launch(name, dev, stream, lambda st: call(at, size, st))
    return workspace


def ssd_linear_attn_varlen_fwd_inplace(o, q, k, v, log_decay, pool, query_start_loc, has_initial_state,
                                       cache_indices, *, scale=None, workspace=None, stream=None):
    """Linear attention with a fixed decay per head over a ragged batch, pool
    updated in place (see include/ssd.h).

    Tensors (torch, on one HIP device): o, v bf16 [T,H,V]; q, k bf16 [T,G,K]
    (q, k and v may be slices of one projection: dense heads, a stride between
    tokens that is a multiple of 8); log_decay fp32 [H]; pool fp32 or bf16
    [S,H,V,K] (updated in place); query_start_loc int32 [batch+1] (rows behind
    the last sequence are left alone); has_initial_state uint8/bool [batch] or
    None; cache_indices int32/uint32 [batch], S or more (or negative) for a
    padding entry.  ``scale``: None for K ** -0.5.  Runs on ``stream`` or the
    current stream; asynchronous.  Returns the workspace tensor (None where none
    is needed).
    """
    batch = query_start_loc.numel() - 1
    slots = pool.shape[0]
    prob, need, dev, state, inputs = _linear_attn(q, k, v, log_decay, batch, slots, _state_dtype(pool, "pool"), scale,
                                                  False)
    out = _dense(o, "o", torch.bfloat16, v.shape, dev)
    states = _dense(pool, "pool", pool.dtype, (slots, *state), dev)
    qsl = _dense(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    idx, flags = _slots(cache_indices, has_initial_state, batch, dev)
    f = load_library().ssd_linear_attn_varlen_fwd_inplace
    return _run("ssd_linear_attn_varlen_fwd_inplace", dev, stream, need, workspace, lambda ws, n, st: f(
        prob, out, *inputs, states, qsl, flags, idx, ws, n, st))


def ssd_linear_attn_varlen_fwd(o, q, k, v, log_decay, initial_states, final_states, query_start_loc, *, scale=None,
                               workspace=None, stream=None):
    """The same with separate states: sequence b starts from
    ``initial_states[b]`` ([batch,H,V,K], or None or empty for zero) and leaves
    ``final_states[b]``; both fp32 or both bf16.  Returns the workspace tensor.
    """
    batch = query_start_loc.numel() - 1
    if final_states is None:
        raise ValueError("final_states is required")
    prob, need, dev, state, inputs = _linear_attn(q, k, v, log_decay, batch, max(batch, 1),
                                                  _state_dtype(final_states, "final_states"), scale, False)
    out = _dense(o, "o", torch.bfloat16, v.shape, dev)
    first = _dense_or_none(initial_states, "initial_states", final_states.dtype, (batch, *state), dev)
    last = _dense(final_states, "final_states", final_states.dtype, (batch, *state), dev)
    qsl = _dense(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    f = load_library().ssd_linear_attn_varlen_fwd
    return _run("ssd_linear_attn_varlen_fwd", dev, stream, need, workspace, lambda ws, n, st: f(
        prob, out, *inputs, first, last, qsl, ws, n, st))


def ssd_linear_attn_varlen_bwd(dq, dk, dv, d_initial_states, q, k, v, d_o, log_decay, initial_states,
                               d_final_states, query_start_loc, *, scale=None, workspace=None, stream=None):
    """Backward pass of ssd_linear_attn_varlen_fwd (see include/ssd.h): dq, dk
    bf16 [T,G,K] and dv bf16 [T,H,V] are written, and ``d_initial_states``
    where it is not None; ``initial_states`` and ``d_final_states`` may be None
    or empty (zero).  State tensors [batch,H,V,K], all fp32 or all bf16.  Returns the
    workspace tensor.
    """
    batch = query_start_loc.numel() - 1
    given = [None if t is None or t.numel() == 0 else t for t in (initial_states, d_final_states)]
    states = ((d_initial_states, "d_initial_states"), (given[0], "initial_states"), (given[1], "d_final_states"))
    kind = next((t for t in states if t[0] is not None), None)
    prob, need, dev, state, inputs = _linear_attn(q, k, v, log_decay, batch, max(batch, 1),
                                                  STATE_F32 if kind is None else _state_dtype(*kind), scale, True)
    d_first, first, d_last = (None if t is None else _dense(t, n, kind[0].dtype, (batch, *state), dev)
                              for t, n in states)
    bf16 = torch.bfloat16
    out = [_dense(dq, "dq", bf16, q.shape, dev), _dense(dk, "dk", bf16, k.shape, dev),
           _dense(dv, "dv", bf16, v.shape, dev)]
    grad = _dense(d_o, "d_o", bf16, v.shape, dev)
    qsl = _dense(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    f = load_library().ssd_linear_attn_varlen_bwd
    return _run("ssd_linear_attn_varlen_bwd", dev, stream, need, workspace, lambda ws, n, st: f(
        prob, *out, d_first, *inputs[:3], grad, inputs[3], first, d_last, qsl, ws, n, st))


def ssd_linear_attn_step_inplace(o, q, k, v, log_decay, pool, has_initial_state, cache_indices, *, scale=None,
                                 stream=None):
    """One token per sequence by the recurrence, pool updated in place (see
    include/ssd.h): row b of o, q, k, v is sequence b's token; other arguments
    as for ssd_linear_attn_varlen_fwd_inplace.  One kernel, no workspace.
    """
    batch = v.shape[0]
    slots = pool.shape[0]
    prob, _, dev, state, inputs = _linear_attn(q, k, v, log_decay, batch, slots, _state_dtype(pool, "pool"), scale,
                                               None)
    out = _dense(o, "o", torch.bfloat16, v.shape, dev)
    states = _dense(pool, "pool", pool.dtype, (slots, *state), dev)
    idx, flags = _slots(cache_indices, has_initial_state, batch, dev)
    f = load_library().ssd_linear_attn_step_inplace
    _launch("ssd_linear_attn_step_inplace", dev, stream, lambda st: f(
        prob, out, *inputs, states, flags, idx, st))


@functools.lru_cache(maxsize=256)
def _state_cache_sizes(*sizes):
    return ctypes.byref(ssd_state_cache_problem(*sizes))


def _state_cache(pool, codes, scales, pool_indices, entry_indices):
    """Problem, device and addresses (pool, codes, scales, pool_indices, entry_indices) of a state-cache call,
    its tensors checked."""
    if torch is None:
        _import_torch()
    dev = pool.device
    if dev.type != "cuda":
        raise ValueError("libssd runs on a HIP device; got tensors on " + str(dev))
    if pool.dim() != 4:
        raise ValueError("pool must be [slots, H, P, N]")
    S, H, P, N = pool.shape
    if codes.dtype == torch.int8:
        form = CODE_I8
    elif codes.dtype == torch.float8_e4m3fn:
        form = CODE_E4M3
    else:
        raise TypeError(f"codes: expected int8 or float8_e4m3fn, got {codes.dtype}")
    E, n = codes.shape[0], pool_indices.numel()
    for t, name in ((pool_indices, "pool_indices"), (entry_indices, "entry_indices")):
        if t.dtype not in (torch.int32, torch.uint32):
            raise TypeError(f"{name} must be int32 or uint32")
    prob = _state_cache_sizes(n, H, P, N, S, E, _state_dtype(pool, "pool"), form)
    return prob, dev, (_dense(pool, "pool", pool.dtype, (S, H, P, N), dev),
                       _dense(codes, "codes", codes.dtype, (E, H, P, N), dev),
                       _dense(scales, "scales", torch.float32, (E, H, P), dev),
                       _dense(pool_indices, "pool_indices", pool_indices.dtype, (n,), dev),
                       _dense(entry_indices, "entry_indices", entry_indices.dtype, (n,), dev))


def ssd_state_quantize(codes, scales, pool, pool_indices, entry_indices, *, stream=None):
    """Park pool slots in 8 bits: slot pool_indices[i] of ``pool`` (fp32 or
    bf16 [S,H,P,N], of the scan or of linear attention) becomes entry
    entry_indices[i] of ``codes`` (int8 or float8_e4m3fn [E,H,P,N]) and
    ``scales`` (fp32 [E,H,P]).  A pair with an index out of range is skipped.
    """
    prob, dev, (p, c, f, i, j) = _state_cache(pool, codes, scales, pool_indices, entry_indices)
    fn = load_library().ssd_state_quantize
    _launch("ssd_state_quantize", dev, stream, lambda st: fn(prob, c, f, p, i, j, st))


def ssd_state_dequantize(pool, codes, scales, pool_indices, entry_indices, *, stream=None):
    """Read parked states back: slot pool_indices[i] of ``pool`` becomes entry
    entry_indices[i] of ``codes`` times its scales."""
    prob, dev, (p, c, f, i, j) = _state_cache(pool, codes, scales, pool_indices, entry_indices)
    fn = load_library().ssd_state_dequantize
    _launch("ssd_state_dequantize", dev, stream, lambda st: fn(prob, p, c, f, i, j, st))


# ---------------------------------------------------------------------------
# the norm, the short convolution and the selective scan, checked in the same way

def ssd_rms_norm_workspace_size(prob: ssd_norm_problem) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_rms_norm_workspace_size(ctypes.byref(prob), ctypes.byref(n)),
           "ssd_rms_norm_workspace_size")
    return n.value


def ssd_causal_conv_workspace_size(prob: ssd_conv_problem) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_causal_conv_workspace_size(ctypes.byref(prob), ctypes.byref(n)),
           "ssd_causal_conv_workspace_size")
    return n.value


def ssd_selective_scan_workspace_size(prob: ssd_selective_problem, backward=False) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_selective_scan_workspace_size(ctypes.byref(prob), 1 if backward else 0,
                                                            ctypes.byref(n)), "ssd_selective_scan_workspace_size")
    return n.value


@functools.lru_cache(maxsize=256)
def _norm_sizes(backward, *sizes):
    prob = ssd_norm_problem(*sizes)
    return ctypes.byref(prob), ssd_rms_norm_workspace_size(prob) if backward else 0


@functools.lru_cache(maxsize=256)
def _conv_sizes(backward, *sizes):
    prob = ssd_conv_problem(*sizes)
    return ctypes.byref(prob), ssd_causal_conv_workspace_size(prob) if backward else 0


@functools.lru_cache(maxsize=256)
def _selective_sizes(backward, *sizes):
    """``backward`` None: of single tokens, which need no workspace and have wider limits"""
    prob = ssd_selective_problem(*sizes)
    return ctypes.byref(prob), 0 if backward is None else ssd_selective_scan_workspace_size(prob, backward)


def _hip_device(t, name, dims):
    if torch is None:
        _import_torch()
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dim() != len(dims):
        raise ValueError(f"{name} must be [{', '.join(dims)}]")
    if t.device.type != "cuda":
        raise ValueError("libssd runs on a HIP device; got tensors on " + str(t.device))
    return t.device


def _row_stride(t, name, shape, device, step):
    """Elements between the rows of a bf16 tensor whose rows are dense (a slice of a wider projection is one), a
    multiple of ``step``; 0 for a dense tensor."""
    if t is None or t.dtype != torch.bfloat16 or t.shape != shape or t.device != device:
        _refuse_tensor(t, name, torch.bfloat16, shape, device)
    if t.is_contiguous():
        return 0
    row = 1
    for n, s in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n > 1 and s != row:
            raise ValueError(f"{name}: the elements of a row must be dense")
        row *= n
    if shape[0] > 1 and (t.stride(0) < row or t.stride(0) % step != 0):
        raise ValueError(f"{name}: the stride between rows must be a multiple of {step} elements, at least {row}")
    return t.stride(0) if shape[0] > 1 else 0


def ssd_rms_norm_fwd(y, scales, residual_out, x, residual, weight, *, eps=1e-5, stream=None):
    """Root-mean-square norm with the residual's addition (see include/ssd.h):
    r = residual + x, y = r / sqrt(mean(r^2) + eps) * weight.

    x bf16 [rows,width] (rows may have a stride, a multiple of 8); residual and
    residual_out fp32 or bf16 [rows,width] (one buffer will do), or both None;
    weight fp32 [width].  y bf16 with ``scales`` None, or int8 or
    float8_e4m3fn codes with ``scales`` fp32 [rows].
    """
    dev = _hip_device(x, "x", ("rows", "width"))
    shape = rows, width = x.shape
    kinds = {torch.bfloat16: OUT_BF16, torch.int8: CODE_I8, torch.float8_e4m3fn: CODE_E4M3}
    if y is None or y.dtype not in kinds:
        raise TypeError("y: expected bfloat16, int8 or float8_e4m3fn, got " + str(None if y is None else y.dtype))
    form = kinds[y.dtype]
    if (scales is None) != (form == OUT_BF16):
        raise ValueError("scales go with 8-bit codes, and with them only")
    if (residual is None) != (residual_out is None):
        raise ValueError("residual and residual_out go together")
    kind = STATE_BF16 if residual is None else _state_dtype(residual, "residual")
    prob, _ = _norm_sizes(False, rows, width, kind, form, float(eps), _row_stride(x, "x", shape, dev, 8))
    out = _dense(y, "y", y.dtype, shape, dev)
    s = None if scales is None else _dense(scales, "scales", torch.float32, (rows,), dev)
    r = r_out = None
    if residual is not None:
        r = _dense(residual, "residual", residual.dtype, shape, dev)
        r_out = _dense(residual_out, "residual_out", residual.dtype, shape, dev)
    w = _dense(weight, "weight", torch.float32, (width,), dev)
    f = load_library().ssd_rms_norm_fwd
    _launch("ssd_rms_norm_fwd", dev, stream, lambda st: f(prob, out, s, r_out, x.data_ptr(), r, w, st))


def ssd_rms_norm_bwd(dx, d_residual, dweight, r, weight, d_y, d_r, *, eps=1e-5, workspace=None, stream=None):
    """Backward pass of ssd_rms_norm_fwd with y in bf16 (see include/ssd.h):
    dx bf16 [rows,width], d_residual (the type of ``r``, or None: dx serves both
    where that is bf16) and dweight fp32 [width] are written.  ``r`` is the forward
    pass's residual_out (its x where there was no residual), ``d_r`` the gradient
    of residual_out or None.  Returns the workspace tensor.
    """
    dev = _hip_device(r, "r", ("rows", "width"))
    shape = rows, width = r.shape
    kind = _state_dtype(r, "r")
    prob, need = _norm_sizes(True, rows, width, kind, OUT_BF16, float(eps), 0)
    out = _dense(dx, "dx", torch.bfloat16, shape, dev)
    d_res = None if d_residual is None else _dense(d_residual, "d_residual", r.dtype, shape, dev)
    dw = _dense(dweight, "dweight", torch.float32, (width,), dev)
    a = _dense(r, "r", r.dtype, shape, dev)
    w = _dense(weight, "weight", torch.float32, (width,), dev)
    g = _dense(d_y, "d_y", torch.bfloat16, shape, dev)
    gr = None if d_r is None else _dense(d_r, "d_r", r.dtype, shape, dev)
    f = load_library().ssd_rms_norm_bwd
    return _run("ssd_rms_norm_bwd", dev, stream, need, workspace, lambda ws, n, st: f(
        prob, out, d_res, dw, a, w, g, gr, ws, n, st))


def _causal_conv(x, weight, bias, batch, slots, silu, backward):
    """Problem and workspace bytes of a convolution call, device, shape of a state, addresses of x, weight and bias."""
    dev = _hip_device(x, "x", ("T", "channels"))
    T, D = x.shape
    if weight is None or weight.dim() != 2:
        raise ValueError("weight must be [channels, width]")
    W = weight.shape[1]
    prob, need = _conv_sizes(backward, T, batch, D, W, slots, 1 if silu else 0, _row_stride(x, "x", (T, D), dev, 8))
    w = _dense(weight, "weight", torch.float32, (D, W), dev)
    b = None if bias is None else _dense(bias, "bias", torch.float32, (D,), dev)
    return prob, need, dev, (W - 1, D), (x.data_ptr(), w, b)


def ssd_causal_conv_varlen_fwd_inplace(y, x, weight, bias, pool, query_start_loc, has_initial_state, cache_indices, *,
                                       silu=True, stream=None):
    """Short causal depthwise convolution over a ragged batch, pool of last
    inputs updated in place (see include/ssd.h).

    y, x bf16 [T,channels] (x may be a slice of a projection: a stride between
    tokens that is a multiple of 8); weight fp32 [channels,width], width 2 to 4;
    bias fp32 [channels] or None; pool bf16 [S,width-1,channels];
    query_start_loc, has_initial_state and cache_indices as for
    ssd_linear_attn_varlen_fwd_inplace.  y may not overlap x.
    """
    batch, slots = query_start_loc.numel() - 1, pool.shape[0]
    prob, _, dev, state, inputs = _causal_conv(x, weight, bias, batch, slots, silu, False)
    out = _dense(y, "y", torch.bfloat16, x.shape, dev)
    states = _dense(pool, "pool", torch.bfloat16, (slots, *state), dev)
    qsl = _dense(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    idx, flags = _slots(cache_indices, has_initial_state, batch, dev)
    f = load_library().ssd_causal_conv_varlen_fwd_inplace
    _launch("ssd_causal_conv_varlen_fwd_inplace", dev, stream, lambda st: f(
        prob, out, *inputs, states, qsl, flags, idx, st))


def ssd_causal_conv_varlen_fwd(y, x, weight, bias, initial_states, final_states, query_start_loc, *, silu=True,
                               stream=None):
    """The same with separate states bf16 [batch,width-1,channels]: sequence b
    follows ``initial_states[b]`` (None or empty: zeros) and leaves
    ``final_states[b]``."""
    batch = query_start_loc.numel() - 1
    prob, _, dev, state, inputs = _causal_conv(x, weight, bias, batch, max(batch, 1), silu, False)
    out = _dense(y, "y", torch.bfloat16, x.shape, dev)
    first = _dense_or_none(initial_states, "initial_states", torch.bfloat16, (batch, *state), dev)
    last = _dense(final_states, "final_states", torch.bfloat16, (batch, *state), dev)
    qsl = _dense(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    f = load_library().ssd_causal_conv_varlen_fwd
    _launch("ssd_causal_conv_varlen_fwd", dev, stream, lambda st: f(prob, out, *inputs, first, last, qsl, st))


def ssd_causal_conv_varlen_bwd(dx, dweight, dbias, d_initial_states, x, weight, bias, d_y, initial_states,
                               d_final_states, query_start_loc, *, silu=True, workspace=None, stream=None):
    """Backward pass of ssd_causal_conv_varlen_fwd (see include/ssd.h): dx bf16
    [T,channels], dweight fp32 [channels,width], dbias fp32 [channels] (or None)
    and ``d_initial_states`` (or None) are written.  Returns the workspace tensor.
    """
    batch = query_start_loc.numel() - 1
    prob, need, dev, state, inputs = _causal_conv(x, weight, bias, batch, max(batch, 1), silu, True)
    bf16, f32 = torch.bfloat16, torch.float32
    out = _dense(dx, "dx", bf16, x.shape, dev)
    dw = _dense(dweight, "dweight", f32, weight.shape, dev)
    db = None if dbias is None else _dense(dbias, "dbias", f32, (x.shape[1],), dev)
    d_first = None if d_initial_states is None else _dense(d_initial_states, "d_initial_states", bf16,
                                                           (batch, *state), dev)
    g = _dense(d_y, "d_y", bf16, x.shape, dev)
    first = _dense_or_none(initial_states, "initial_states", bf16, (batch, *state), dev)
    d_last = _dense_or_none(d_final_states, "d_final_states", bf16, (batch, *state), dev)
    qsl = _dense(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    f = load_library().ssd_causal_conv_varlen_bwd
    return _run("ssd_causal_conv_varlen_bwd", dev, stream, need, workspace, lambda ws, n, st: f(
        prob, out, dw, db, d_first, *inputs, g, first, d_last, qsl, ws, n, st))


def ssd_causal_conv_step_inplace(y, x, weight, bias, pool, has_initial_state, cache_indices, *, silu=True,
                                 stream=None):
    """One token per sequence (see include/ssd.h): row b of y and x is sequence
    b's token; other arguments as for ssd_causal_conv_varlen_fwd_inplace."""
    batch, slots = x.shape[0], pool.shape[0]
    prob, _, dev, state, inputs = _causal_conv(x, weight, bias, batch, slots, silu, False)
    out = _dense(y, "y", torch.bfloat16, x.shape, dev)
    states = _dense(pool, "pool", torch.bfloat16, (slots, *state), dev)
    idx, flags = _slots(cache_indices, has_initial_state, batch, dev)
    f = load_library().ssd_causal_conv_step_inplace
    _launch("ssd_causal_conv_step_inplace", dev, stream, lambda st: f(prob, out, *inputs, states, flags, idx, st))


def _selective(x, dt, A, B, C, D, z, dt_bias, batch, slots, state_dtype, dt_softplus, backward):
    """Problem and workspace bytes of a selective-scan call, device, shape of a state, addresses of x, dt, A, B, C,
    D, z and dt_bias."""
    dev = _hip_device(x, "x", ("T", "channels"))
    tokens = T, ch = x.shape
    if B is None or B.dim() != 3:
        raise ValueError("B must be [T, groups, dstate]")
    _, G, N = bc = B.shape
    if bc[0] != T:
        _refuse_tensor(B, "B", torch.bfloat16, (T, G, N), dev)
    prob, need = _selective_sizes(
        backward, T, batch, ch, G, N, slots, 1 if dt_softplus else 0, state_dtype,
        _row_stride(x, "x", tokens, dev, 8), _row_stride(dt, "dt", tokens, dev, 8),
        0 if z is None else _row_stride(z, "z", tokens, dev, 8), _row_stride(B, "B", bc, dev, 2),
        _row_stride(C, "C", bc, dev, 2))
    f32 = torch.float32
    return prob, need, dev, (ch, N), (
        x.data_ptr(), dt.data_ptr(), _dense(A, "A", f32, (ch, N), dev), B.data_ptr(), C.data_ptr(),
        None if D is None else _dense(D, "D", f32, (ch,), dev), None if z is None else z.data_ptr(),
        None if dt_bias is None else _dense(dt_bias, "dt_bias", f32, (ch,), dev))


def ssd_selective_scan_varlen_fwd_inplace(y, x, dt, A, B, C, D, z, dt_bias, pool, query_start_loc, has_initial_state,
                                          cache_indices, *, dt_softplus=True, workspace=None, stream=None):
    """Selective scan (a decay per channel and state) over a ragged batch, pool
    updated in place (see include/ssd.h).

    y bf16 [T,channels]; x, dt, z bf16 [T,channels] and B, C bf16 [T,G,N]
    (slices of projections will do: a stride between tokens that is a multiple of
    8, of B and C even); A fp32 [channels,N]; D, dt_bias fp32 [channels] or None;
    z None for no gate; pool fp32 or bf16 [S,channels,N]; query_start_loc,
    has_initial_state and cache_indices as for
    ssd_linear_attn_varlen_fwd_inplace.  Returns the workspace tensor (None where
    none is needed).
    """
    batch, slots = query_start_loc.numel() - 1, pool.shape[0]
    prob, need, dev, state, inputs = _selective(x, dt, A, B, C, D, z, dt_bias, batch, slots,
                                                _state_dtype(pool, "pool"), dt_softplus, False)
    out = _dense(y, "y", torch.bfloat16, x.shape, dev)
    states = _dense(pool, "pool", pool.dtype, (slots, *state), dev)
    qsl = _dense(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    idx, flags = _slots(cache_indices, has_initial_state, batch, dev)
    f = load_library().ssd_selective_scan_varlen_fwd_inplace
    return _run("ssd_selective_scan_varlen_fwd_inplace", dev, stream, need, workspace, lambda ws, n, st: f(
        prob, out, *inputs, states, qsl, flags, idx, ws, n, st))


def ssd_selective_scan_varlen_fwd(y, x, dt, A, B, C, D, z, dt_bias, initial_states, final_states, query_start_loc, *,
                                  dt_softplus=True, workspace=None, stream=None):
    """The same with separate states [batch,channels,N]: sequence b starts from
    ``initial_states[b]`` (None or empty: zero) and leaves ``final_states[b]``;
    both fp32 or both bf16.  Returns the workspace tensor."""
    batch = query_start_loc.numel() - 1
    if final_states is None:
        raise ValueError("final_states is required")
    prob, need, dev, state, inputs = _selective(x, dt, A, B, C, D, z, dt_bias, batch, max(batch, 1),
                                                _state_dtype(final_states, "final_states"), dt_softplus, False)
    out = _dense(y, "y", torch.bfloat16, x.shape, dev)
    first = _dense_or_none(initial_states, "initial_states", final_states.dtype, (batch, *state), dev)
    last = _dense(final_states, "final_states", final_states.dtype, (batch, *state), dev)
    qsl = _dense(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    f = load_library().ssd_selective_scan_varlen_fwd
    return _run("ssd_selective_scan_varlen_fwd", dev, stream, need, workspace, lambda ws, n, st: f(
        prob, out, *inputs, first, last, qsl, ws, n, st))


def ssd_selective_scan_varlen_bwd(dx, ddt, dA, dB, dC, dD, dz, ddt_bias, d_initial_states, x, dt, A, B, C, D, z,
                                  dt_bias, d_y, initial_states, d_final_states, query_start_loc, *, dt_softplus=True,
                                  workspace=None, stream=None):
    """Backward pass of ssd_selective_scan_varlen_fwd (see include/ssd.h): dx,
    ddt, dz bf16 [T,channels] (dz None where z is), dB, dC bf16 [T,G,N], dA fp32
    [channels,N] are written, and dD, ddt_bias fp32 [channels] and
    ``d_initial_states`` where they are not None.  State tensors
    [batch,channels,N], all fp32 or all bf16.  Returns the workspace tensor.
    """
    batch = query_start_loc.numel() - 1
    given = [None if t is None or t.numel() == 0 else t for t in (initial_states, d_final_states)]
    states = ((d_initial_states, "d_initial_states"), (given[0], "initial_states"), (given[1], "d_final_states"))
    kind = next((t for t in states if t[0] is not None), None)
    prob, need, dev, state, inputs = _selective(x, dt, A, B, C, D, z, dt_bias, batch, max(batch, 1),
                                                STATE_F32 if kind is None else _state_dtype(*kind), dt_softplus, True)
    if (z is None) != (dz is None):
        raise ValueError("dz goes with z, and with it only")
    d_first, first, d_last = (None if t is None else _dense(t, n, kind[0].dtype, (batch, *state), dev)
                              for t, n in states)
    bf16, f32 = torch.bfloat16, torch.float32
    rows, ch = [None if t is None else _dense(t, n, bf16, x.shape, dev)
                for t, n in ((dx, "dx"), (ddt, "ddt"), (dz, "dz"))], (x.shape[1],)
    if dx is None or ddt is None:
        raise ValueError("dx and ddt are required")
    a = _dense(dA, "dA", f32, A.shape, dev)
    b, c = (_dense(t, n, bf16, B.shape, dev) for t, n in ((dB, "dB"), (dC, "dC")))
    d, e = (None if t is None else _dense(t, n, f32, ch, dev) for t, n in ((dD, "dD"), (ddt_bias, "ddt_bias")))
    g = _dense(d_y, "d_y", bf16, x.shape, dev)
    qsl = _dense(query_start_loc, "query_start_loc", torch.int32, (batch + 1,), dev)
    f = load_library().ssd_selective_scan_varlen_bwd
    return _run("ssd_selective_scan_varlen_bwd", dev, stream, need, workspace, lambda ws, n, st: f(
        prob, rows[0], rows[1], a, b, c, d, rows[2], e, d_first, *inputs, g, first, d_last, qsl, ws, n, st))


def ssd_selective_scan_step_inplace(y, x, dt, A, B, C, D, z, dt_bias, pool, has_initial_state, cache_indices, *,
                                    dt_softplus=True, stream=None):
    """One token per sequence by the recurrence (see include/ssd.h): row b of y,
    x, dt, B, C, z is sequence b's token; other arguments as for
    ssd_selective_scan_varlen_fwd_inplace.  One kernel, no workspace."""
    batch, slots = x.shape[0], pool.shape[0]
    prob, _, dev, state, inputs = _selective(x, dt, A, B, C, D, z, dt_bias, batch, slots,
                                             _state_dtype(pool, "pool"), dt_softplus, None)
    out = _dense(y, "y", torch.bfloat16, x.shape, dev)
    states = _dense(pool, "pool", pool.dtype, (slots, *state), dev)
    idx, flags = _slots(cache_indices, has_initial_state, batch, dev)
    f = load_library().ssd_selective_scan_step_inplace
    _launch("ssd_selective_scan_step_inplace", dev, stream, lambda st: f(prob, out, *inputs, states, flags, idx, st))
