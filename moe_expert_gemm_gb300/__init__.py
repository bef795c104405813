"""Fused MoE expert GEMM + EP-combine send for GB300 (sm_103a).

Python binding of the C ABI in ``include/moe_ep.h`` (``libmoe_ep.so``), with the
same entry-point names. It only marshals arguments: pointers are plain integers
(or objects with ``data_ptr()``), streams are ``cudaStream_t`` handles (or
objects with ``cuda_stream``). Every step of the path runs in the library's
kernels; there is no fallback, and a missing library raises.
"""

from __future__ import annotations

import ctypes
import os

from .build import LIB_PATH, build  # noqa: F401

EP_MAX_RANKS = 8
EP_MAX_LOCAL_EXPERTS = 256

EP_OK = 0
EP_ERR_INVALID_ARG = -1
EP_ERR_UNSUPPORTED = -2
EP_ERR_CUDA = -3

EP_STATUS_BOUNDS = 0x1
EP_STATUS_TIMEOUT = 0x2
EP_STATUS_CAPACITY = 0x4
EP_ACT_NONE = 0
EP_ACT_SWIGLU = 1
EP_SIGNAL_RANK_FLAG = 0
EP_SIGNAL_PER_EXPERT = 1
EP_OVERLAP_NONE = 0
EP_OVERLAP_ANY = 1
EP_OVERLAP_INPUTS_READY = 2
EP_STATUS_ROUTING = 0x8
EP_STATUS_INTERNAL = 0x10

EP_BF16 = 0
EP_FP8_1D2D = 1

EP_SCORE_SOFTMAX = 0
EP_SCORE_SIGMOID = 1
EP_LOGITS_F32 = 0
EP_LOGITS_BF16 = 1
EP_W4_INT = 0
EP_W4_E2M1 = 1
EP_ROWS_F32 = 0
EP_ROWS_BF16 = 1
EP_MAX_NORM_HIDDEN = 16384
EP_MAX_FEW_TOKENS = 64
EP_FEW_COUNTER_BYTES = 4096

_c_i32, _c_i64, _c_u64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p


class ep_config(ctypes.Structure):
    _fields_ = [(n, _c_i32) for n in ("n_ranks", "my_rank", "n_local_experts", "top_k",
                                      "num_tokens", "max_tokens_per_rank", "K", "N",
                                      "msg_bytes", "dtype", "send_warps", "signal_mode")]


class ep_plan_out(ctypes.Structure):
    _fields_ = [("expert_offsets", _vp), ("src_info", _vp), ("seg_offsets", _vp),
                ("send_counts", _vp), ("gather_idx", _vp), ("m_total", _vp), ("status", _vp),
                ("max_rows", _c_i64)]


class ep_send_args(ctypes.Structure):
    _fields_ = [("A", _vp), ("a_scales", _vp), ("W", _vp), ("w_scales", _vp),
                ("expert_offsets", _vp), ("src_info", _vp), ("seg_offsets", _vp),
                ("send_counts", _vp), ("max_rows", _c_i64),
                ("recv_buf_ptrs", _vp * EP_MAX_RANKS), ("recv_count_ptrs", _vp * EP_MAX_RANKS),
                ("atomic_counter", _vp), ("rank_completion_counter", _vp), ("epoch", _c_u64),
                ("p3_control", _c_i32), ("C", _vp), ("status", _vp), ("trace", _vp),
                ("timeout_ns", _c_i64), ("trace_records", _c_i64),
                ("local_activation", _c_i32), ("overlap_previous", _c_i32)]


class ep_combine_args(ctypes.Structure):
    _fields_ = [("recv_buf", _vp), ("recv_count", _vp), ("gates", _vp), ("out", _vp),
                ("epoch", _c_u64), ("timeout_ns", _c_i64), ("status", _vp),
                ("topk_ids", _vp), ("overlap_previous", _c_i32)]


class ep_scatter_args(ctypes.Structure):
    _fields_ = [("C", _vp), ("expert_offsets", _vp), ("src_info", _vp), ("seg_offsets", _vp),
                ("send_counts", _vp), ("max_rows", _c_i64),
                ("recv_buf_ptrs", _vp * EP_MAX_RANKS), ("recv_count_ptrs", _vp * EP_MAX_RANKS),
                ("block_counter", _vp), ("epoch", _c_u64), ("status", _vp)]


class ep_dispatch_args(ctypes.Structure):
    _fields_ = [("x_ptrs", _vp * EP_MAX_RANKS), ("gather_idx", _vp), ("expert_offsets", _vp),
                ("max_rows", _c_i64), ("hidden", _c_i32), ("A_in", _vp), ("status", _vp)]


class ep_swiglu_args(ctypes.Structure):
    _fields_ = [("G", _vp), ("A", _vp), ("expert_offsets", _vp), ("max_rows", _c_i64),
                ("inter", _c_i32)]


class ep_route_args(ctypes.Structure):
    _fields_ = [("logits", _vp), ("logits_stride", _c_i64), ("logits_dtype", _c_i32),
                ("score", _c_i32), ("bias", _vp), ("n_groups", _c_i32), ("topk_groups", _c_i32),
                ("group_top", _c_i32), ("renormalize", _c_i32), ("scale", ctypes.c_float),
                ("topk_ids", _vp), ("gates", _vp)]


class ep_route_backward_args(ctypes.Structure):
    _fields_ = [("logits", _vp), ("logits_stride", _c_i64), ("logits_dtype", _c_i32),
                ("score", _c_i32), ("renormalize", _c_i32), ("scale", ctypes.c_float),
                ("topk_ids", _vp), ("dgates", _vp), ("dlogits", _vp),
                ("dlogits_stride", _c_i64), ("status", _vp)]


class ep_combine_backward_args(ctypes.Structure):
    _fields_ = [("recv_buf", _vp), ("gates", _vp), ("dout", _vp), ("dgates", _vp),
                ("drows", _vp)]


class ep_w4_args(ctypes.Structure):
    _fields_ = [("A", _vp), ("x_ptrs", _vp * EP_MAX_RANKS), ("gather_idx", _vp), ("W", _vp),
                ("w_scales", _vp), ("w_zeros", _vp), ("w_format", _c_i32),
                ("group_size", _c_i32), ("expert_offsets", _vp), ("max_rows", _c_i64),
                ("local_activation", _c_i32), ("C", _vp), ("workspace", _vp),
                ("workspace_bytes", _c_i64), ("status", _vp)]


class ep_add_rmsnorm_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_stride", _c_i64), ("residual", _vp), ("residual_stride", _c_i64),
                ("residual_dtype", _c_i32), ("weight_dtype", _c_i32), ("weight", _vp),
                ("eps", ctypes.c_float), ("hidden", _c_i32), ("sum", _vp), ("sum_stride", _c_i64),
                ("y", _vp), ("y_stride", _c_i64), ("q", _vp), ("q_scales", _vp)]


class ep_add_rmsnorm_backward_args(ctypes.Structure):
    _fields_ = [("h", _vp), ("h_stride", _c_i64), ("h_dtype", _c_i32), ("weight_dtype", _c_i32),
                ("dy", _vp), ("dy_stride", _c_i64), ("dsum", _vp), ("dsum_stride", _c_i64),
                ("weight", _vp), ("eps", ctypes.c_float), ("hidden", _c_i32), ("dh", _vp),
                ("dh_stride", _c_i64), ("dx", _vp), ("dx_stride", _c_i64), ("dweight", _vp),
                ("workspace", _vp), ("workspace_bytes", _c_i64)]


class ep_swiglu_e4m3_args(ctypes.Structure):
    _fields_ = [("G", _vp), ("q", _vp), ("q_scales", _vp), ("expert_offsets", _vp),
                ("max_rows", _c_i64), ("inter", _c_i32)]


class ep_layer_few_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_scales", _vp), ("topk_ids", _vp), ("gates", _vp), ("W1", _vp),
                ("w1_scales", _vp), ("W2", _vp), ("w2_scales", _vp), ("out", _vp),
                ("workspace", _vp), ("workspace_bytes", _c_i64), ("status", _vp),
                ("timeout_ns", _c_i64)]


EP_IPC_HANDLE_BYTES = 64


class ep_ipc_handle(ctypes.Structure):
    _fields_ = [("handle", ctypes.c_uint8 * EP_IPC_HANDLE_BYTES), ("offset", _c_u64),
                ("bytes", _c_u64)]


class EpError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {ep_strerror(code)} ({code})")
        self.code = code


_lib = None

EXPORTS = ("ep_plan_sizes", "ep_plan", "grouped_gemm_combine_send", "ep_combine_reduce",
           "ep_strerror", "grouped_gemm_combine_send_noalloc", "ep_scatter_send",
           "ep_dispatch_gather", "ep_swiglu", "ep_ipc_export", "ep_ipc_import", "ep_ipc_close",
           "ep_route", "ep_route_backward", "ep_combine_backward", "ep_matvec_w4_sizes",
           "ep_matvec_w4", "ep_add_rmsnorm", "ep_add_rmsnorm_backward_sizes",
           "ep_add_rmsnorm_backward", "ep_swiglu_e4m3", "ep_layer_few_sizes", "ep_layer_few")


def load(build_if_missing: bool = True):
    """Load libmoe_ep.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing:
        build()
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} not built; run moe_expert_gemm_gb300.build()")
    L = ctypes.CDLL(LIB_PATH)
    L.ep_plan_sizes.argtypes = [ctypes.POINTER(ep_config), ctypes.POINTER(_c_i64)]
    L.ep_plan.argtypes = [ctypes.POINTER(ep_config), _vp, ctypes.POINTER(ep_plan_out), _vp]
    L.grouped_gemm_combine_send.argtypes = [ctypes.POINTER(ep_config),
                                            ctypes.POINTER(ep_send_args), _vp]
    L.ep_combine_reduce.argtypes = [ctypes.POINTER(ep_config), ctypes.POINTER(ep_combine_args),
                                    _vp]
    L.grouped_gemm_combine_send_noalloc.argtypes = [ctypes.POINTER(ep_config),
                                                    ctypes.POINTER(ep_send_args), _vp]
    L.ep_scatter_send.argtypes = [ctypes.POINTER(ep_config), ctypes.POINTER(ep_scatter_args), _vp]
    L.ep_dispatch_gather.argtypes = [ctypes.POINTER(ep_config), ctypes.POINTER(ep_dispatch_args),
                                     _vp]
    L.ep_swiglu.argtypes = [ctypes.POINTER(ep_config), ctypes.POINTER(ep_swiglu_args), _vp]
    L.ep_ipc_export.argtypes = [_vp, ctypes.POINTER(ep_ipc_handle)]
    L.ep_ipc_import.argtypes = [ctypes.POINTER(ep_ipc_handle), ctypes.POINTER(_vp)]
    L.ep_ipc_close.argtypes = [ctypes.POINTER(ep_ipc_handle), _vp]
    for f, args in (("ep_route", ep_route_args), ("ep_route_backward", ep_route_backward_args),
                    ("ep_combine_backward", ep_combine_backward_args),
                    ("ep_matvec_w4", ep_w4_args), ("ep_add_rmsnorm", ep_add_rmsnorm_args),
                    ("ep_add_rmsnorm_backward", ep_add_rmsnorm_backward_args),
                    ("ep_swiglu_e4m3", ep_swiglu_e4m3_args), ("ep_layer_few", ep_layer_few_args)):
        getattr(L, f).argtypes = [ctypes.POINTER(ep_config), ctypes.POINTER(args), _vp]
    for f in ("ep_matvec_w4_sizes", "ep_layer_few_sizes"):
        getattr(L, f).argtypes = [ctypes.POINTER(ep_config), ctypes.POINTER(_c_i64)]
    L.ep_add_rmsnorm_backward_sizes.argtypes = [ctypes.POINTER(ep_config), _c_i32,
                                                ctypes.POINTER(_c_i64)]
    for f in ("ep_plan_sizes", "ep_plan", "grouped_gemm_combine_send", "ep_combine_reduce",
              "grouped_gemm_combine_send_noalloc", "ep_scatter_send", "ep_dispatch_gather",
              "ep_swiglu", "ep_ipc_export", "ep_ipc_import", "ep_ipc_close",
              "ep_route", "ep_route_backward", "ep_combine_backward", "ep_matvec_w4_sizes",
              "ep_matvec_w4", "ep_add_rmsnorm", "ep_add_rmsnorm_backward_sizes",
              "ep_add_rmsnorm_backward", "ep_swiglu_e4m3", "ep_layer_few_sizes", "ep_layer_few"):
        getattr(L, f).restype = ctypes.c_int
    L.ep_strerror.argtypes = [ctypes.c_int]
    L.ep_strerror.restype = ctypes.c_char_p
    _lib = L
    return L


def ptr(x) -> int:
    """Device address of a tensor-like object, or the integer itself (None -> 0)."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def stream_handle(s) -> int:
    if s is None:
        return 0
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _check(rc: int, where: str) -> int:
    if rc != EP_OK:
        raise EpError(rc, where)
    return rc


def ep_strerror(code: int) -> str:
    return load().ep_strerror(code).decode()


def ep_plan_sizes(cfg: ep_config) -> int:
    out = _c_i64(0)
    _check(load().ep_plan_sizes(ctypes.byref(cfg), ctypes.byref(out)), "ep_plan_sizes")
    return int(out.value)


def ep_plan(cfg: ep_config, topk_ids, out: ep_plan_out, stream=None) -> int:
    return _check(load().ep_plan(ctypes.byref(cfg), ptr(topk_ids), ctypes.byref(out),
                                 stream_handle(stream)), "ep_plan")


def grouped_gemm_combine_send(cfg: ep_config, args: ep_send_args, stream=None) -> int:
    return _check(load().grouped_gemm_combine_send(ctypes.byref(cfg), ctypes.byref(args),
                                                   stream_handle(stream)),
                  "grouped_gemm_combine_send")


def grouped_gemm_combine_send_noalloc(cfg: ep_config, args: ep_send_args, stream=None) -> int:
    """The fused send for callers that cannot allocate: the counter arrays come
    from the library's own device array (args' counter pointers are ignored)."""
    return _check(load().grouped_gemm_combine_send_noalloc(ctypes.byref(cfg), ctypes.byref(args),
                                                           stream_handle(stream)),
                  "grouped_gemm_combine_send_noalloc")


def ep_scatter_send(cfg: ep_config, args: ep_scatter_args, stream=None) -> int:
    """The send step alone (unfused comparator): local C rows to the receive
    buffers, then the count words and the rank flags."""
    return _check(load().ep_scatter_send(ctypes.byref(cfg), ctypes.byref(args),
                                         stream_handle(stream)), "ep_scatter_send")


def ep_dispatch_gather(cfg: ep_config, args: ep_dispatch_args, stream=None) -> int:
    """Dispatch: every routed token row to its expert's rank, in plan order."""
    return _check(load().ep_dispatch_gather(ctypes.byref(cfg), ctypes.byref(args),
                                            stream_handle(stream)), "ep_dispatch_gather")


def ep_swiglu(cfg: ep_config, args: ep_swiglu_args, stream=None) -> int:
    """A = bf16(SiLU(gate) * up) from the up/gate GEMM's rows."""
    return _check(load().ep_swiglu(ctypes.byref(cfg), ctypes.byref(args),
                                   stream_handle(stream)), "ep_swiglu")


def ep_combine_reduce(cfg: ep_config, args: ep_combine_args, stream=None) -> int:
    return _check(load().ep_combine_reduce(ctypes.byref(cfg), ctypes.byref(args),
                                           stream_handle(stream)), "ep_combine_reduce")


def ep_route(cfg: ep_config, args: ep_route_args, stream=None) -> int:
    """The router: every token's experts (topk_ids) and gates from its logits."""
    return _check(load().ep_route(ctypes.byref(cfg), ctypes.byref(args),
                                  stream_handle(stream)), "ep_route")


def ep_route_backward(cfg: ep_config, args: ep_route_backward_args, stream=None) -> int:
    """Gradient of the gates with respect to the router's logits."""
    return _check(load().ep_route_backward(ctypes.byref(cfg), ctypes.byref(args),
                                           stream_handle(stream)), "ep_route_backward")


def ep_combine_backward(cfg: ep_config, args: ep_combine_backward_args, stream=None) -> int:
    """Gradients of the combine's sum: of the gates, of the combined rows."""
    return _check(load().ep_combine_backward(ctypes.byref(cfg), ctypes.byref(args),
                                             stream_handle(stream)), "ep_combine_backward")


def ep_matvec_w4_sizes(cfg: ep_config) -> int:
    """Workspace bytes of ep_matvec_w4 (zero the workspace before its first use)."""
    out = _c_i64(0)
    _check(load().ep_matvec_w4_sizes(ctypes.byref(cfg), ctypes.byref(out)), "ep_matvec_w4_sizes")
    return int(out.value)


def ep_matvec_w4(cfg: ep_config, args: ep_w4_args, stream=None) -> int:
    """Expert products of a few rows on 4-bit weights with group scales."""
    return _check(load().ep_matvec_w4(ctypes.byref(cfg), ctypes.byref(args),
                                      stream_handle(stream)), "ep_matvec_w4")


def ep_add_rmsnorm(cfg: ep_config, args: ep_add_rmsnorm_args, stream=None) -> int:
    """The residual's addition and the norm in front of a layer, in bf16 or 8 bits with scales."""
    return _check(load().ep_add_rmsnorm(ctypes.byref(cfg), ctypes.byref(args),
                                        stream_handle(stream)), "ep_add_rmsnorm")


def ep_add_rmsnorm_backward_sizes(cfg: ep_config, hidden: int) -> int:
    """Workspace bytes of ep_add_rmsnorm_backward."""
    out = _c_i64(0)
    _check(load().ep_add_rmsnorm_backward_sizes(ctypes.byref(cfg), hidden, ctypes.byref(out)),
           "ep_add_rmsnorm_backward_sizes")
    return int(out.value)


def ep_add_rmsnorm_backward(cfg: ep_config, args: ep_add_rmsnorm_backward_args, stream=None) -> int:
    """Gradients of the norm: of its input (and the residual), of its weight."""
    return _check(load().ep_add_rmsnorm_backward(ctypes.byref(cfg), ctypes.byref(args),
                                                 stream_handle(stream)), "ep_add_rmsnorm_backward")


def ep_swiglu_e4m3(cfg: ep_config, args: ep_swiglu_e4m3_args, stream=None) -> int:
    """SiLU(gate) * up from the up/gate GEMM's rows, as e4m3 rows with 1x128 scales."""
    return _check(load().ep_swiglu_e4m3(ctypes.byref(cfg), ctypes.byref(args),
                                        stream_handle(stream)), "ep_swiglu_e4m3")


def ep_layer_few_sizes(cfg: ep_config) -> int:
    """Workspace bytes of ep_layer_few (zero the first EP_FEW_COUNTER_BYTES before its first use)."""
    out = _c_i64(0)
    _check(load().ep_layer_few_sizes(ctypes.byref(cfg), ctypes.byref(out)), "ep_layer_few_sizes")
    return int(out.value)


def ep_layer_few(cfg: ep_config, args: ep_layer_few_args, stream=None) -> int:
    """A whole MoE layer for a few tokens: the rank's experts' part of their outputs."""
    return _check(load().ep_layer_few(ctypes.byref(cfg), ctypes.byref(args),
                                      stream_handle(stream)), "ep_layer_few")


def ep_ipc_export(dev_ptr) -> ep_ipc_handle:
    """CUDA IPC handle (plus offset) of a device buffer of this process, for the peer
    processes of an expert-parallel group to map (ep_ipc_import)."""
    h = ep_ipc_handle()
    _check(load().ep_ipc_export(ptr(dev_ptr), ctypes.byref(h)), "ep_ipc_export")
    return h


def ep_ipc_import(h: ep_ipc_handle) -> int:
    """Map another process's exported buffer; returns its address in this process."""
    out = _vp(0)
    _check(load().ep_ipc_import(ctypes.byref(h), ctypes.byref(out)), "ep_ipc_import")
    return int(out.value)


def ep_ipc_close(h: ep_ipc_handle, dev_ptr: int) -> int:
    return _check(load().ep_ipc_close(ctypes.byref(h), ptr(dev_ptr)), "ep_ipc_close")


def raw_call(name: str, *args) -> int:
    """Call an entry point and return its code without raising (for error-path tests)."""
    return int(getattr(load(), name)(*args))
