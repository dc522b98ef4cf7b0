"""Thin Python binding of libpi (include/pi.h): same entry-point names,
argument marshalling only.  Every step of the hot path runs in the library's
CUDA kernels; there is no CPU fallback.  If ``_build/libpi.so`` is missing this
module raises on first use -- build it with
``python -m activation_sparse_decode_sigmoid_gb300.build``.

Tensors are torch tensors on the context's device (PyTorch supplies device
memory and streams only).  16-bit data may be passed as float16 / bfloat16 or
as int16 / uint16 views of the bit patterns; the block operators (linear,
gated FFN, norms) take float16, bfloat16 and float32 tensors as they are.  Every
compute call is issued on torch's current CUDA stream.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libpi.so")

PI_OK = 0
PI_ERR_ARG, PI_ERR_SHAPE, PI_ERR_CUDA, PI_ERR_OOM = -1, -2, -3, -4
PI_ERR_NOT_LOADED, PI_ERR_TIMEOUT, PI_ERR_DEVICE_FLAG, PI_ERR_UNSUPPORTED = -5, -6, -7, -8
PI_RELU, PI_REGLU, PI_SQRELU = 0, 1, 2
PI_F16, PI_BF16, PI_Q4_0, PI_F32, PI_MX8, PI_MX4 = range(6)
PI_FN_NONE, PI_FN_RELU, PI_FN_SQRELU, PI_FN_SIGMOID, PI_FN_SILU, PI_FN_GELU, PI_FN_GELU_TANH = range(7)
PI_NORM_NONE, PI_NORM_RMS, PI_NORM_LAYER = 0, 1, 2

# every symbol include/pi.h declares
EXPORTS = ("pi_create", "pi_destroy", "pi_set_stream", "pi_load_layer", "pi_layer_counts",
           "pi_perm_from_counts", "pi_predict", "pi_sparse_ffn", "pi_dense_ffn", "pi_decode_step",
           "pi_decode_step_host",
           "pi_dense_step", "pi_set_trace", "pi_sync_status", "pi_last_error", "pi_grid_size",
           "pi_debug_set_wait_limit", "pi_debug_barrier_extra", "pi_debug_set_timeline",
           "pi_debug_set_tuning", "pi_debug_copy_hidden", "pi_debug_set_mma_min_batch",
           "pi_sparse_ffn_noalloc", "pi_set_hot_prefix", "pi_hot_prefix_crossover", "pi_choose_hot_prefix",
           "pi_layerwise_min_batch", "pi_load_layer_shard", "pi_layer_shard", "pi_layer_partial",
           "pi_residual_add", "pi_linear_workspace", "pi_linear", "pi_linear_bwd", "pi_gated_ffn_workspace",
           "pi_gated_ffn", "pi_gated_ffn_bwd", "pi_norm_residual", "pi_norm_residual_bwd_workspace",
           "pi_norm_residual_bwd", "pi_mx_bytes", "pi_mx_quantize", "pi_mx_dequantize", "pi_mx_linear_workspace",
           "pi_mx_linear", "pi_mx_gated_ffn_workspace", "pi_mx_gated_ffn", "pi_norm_residual_mx")


class PiError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libpi status {status}: {msg}")
        self.status = status


class pi_layer_desc(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_ffn", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("act", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("act_dtype", ctypes.c_int32)]


class pi_ffn_rows(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_ffn", ctypes.c_int32), ("act", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("up", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("down_rows", ctypes.c_void_p), ("b", ctypes.c_void_p), ("b_down", ctypes.c_void_p)]


class pi_layer_weights(ctypes.Structure):
    _fields_ = [("w_up", ctypes.c_void_p), ("w_gate", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("b_down", ctypes.c_void_p), ("p_w1", ctypes.c_void_p),
                ("p_b1", ctypes.c_void_p), ("p_w2", ctypes.c_void_p), ("p_b2", ctypes.c_void_p),
                ("on_device", ctypes.c_int32)]


def _struct(name, i32=(), f32=(), i64=(), ptr=()):
    """A ctypes struct of 32-bit integers, floats, 64-bit integers and
    pointers; f32 maps the names among i32 that are floats."""
    fields = [(n, ctypes.c_float if n in f32 else ctypes.c_int32) for n in i32]
    fields += [(n, ctypes.c_int64) for n in i64] + [(n, ctypes.c_void_p) for n in ptr]
    return type(name, (ctypes.Structure,), {"_fields_": fields})


pi_linear_desc = _struct("pi_linear_desc", ("T", "K", "N", "dtype", "out_dtype", "grad_dtype", "fn", "scale", "unaligned"),
                         ("scale",), ("ldx", "ldw", "ldz", "ldr", "ldy", "lddx", "lddw"))
pi_gated_ffn_desc = _struct("pi_gated_ffn_desc", ("T", "d", "n", "dtype", "grad_dtype", "fn", "gated", "unaligned"), (),
                            ("ldx", "ldy", "ld_gate", "ld_up", "ld_down", "ldg", "ldu", "lda"))
pi_gated_ffn_weights = _struct("pi_gated_ffn_weights", ptr=("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down"))
pi_gated_ffn_save = _struct("pi_gated_ffn_save", ptr=("g", "u", "a"))
pi_gated_ffn_grads = _struct("pi_gated_ffn_grads", ptr=("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down"))
pi_norm_residual_desc = _struct("pi_norm_residual_desc",
                                ("T", "d", "x_dtype", "dtype", "grad_dtype", "pre", "post", "gate_rows", "res_scale",
                                 "branch_scale", "eps"), ("res_scale", "branch_scale", "eps"),
                                ("ldx", "ldxo", "ldy", "ldh", "ldgate", "lddxo"))
pi_norm_residual_params = _struct("pi_norm_residual_params", ptr=("w_pre", "b_pre", "w_post", "b_post"))
pi_norm_residual_grads = _struct("pi_norm_residual_grads",
                                 ptr=("dx", "dy", "dgate", "dw_pre", "db_pre", "dw_post", "db_post"))


_lib = None

pi_mx = _struct("pi_mx", ptr=("codes", "scales"))
pi_mx_desc = _struct("pi_mx_desc", ("rows", "cols", "kind", "dtype"), (), ("ldx", "ldq"))
pi_mx_linear_desc = _struct("pi_mx_linear_desc", ("T", "K", "N", "x_kind", "w_kind", "dtype", "out_dtype", "fn", "scale"),
                            ("scale",), ("ldx", "ldw", "ldr", "ldy"))
pi_mx_gated_ffn_desc = _struct("pi_mx_gated_ffn_desc", ("T", "d", "n", "x_kind", "w_kind", "dtype", "fn", "gated"), (),
                               ("ldx", "ld_gate", "ld_up", "ld_down", "ldy"))
# (the three matrices' pointers one after the other)
pi_mx_gated_ffn_weights = _struct("pi_mx_gated_ffn_weights",
                                  ptr=("gate_codes", "gate_scales", "up_codes", "up_scales", "down_codes", "down_scales",
                                       "b_gate", "b_up", "b_down"))


def load_library(path: str = LIB_PATH):
    """Load libpi.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libpi.so not built ({path}); run python -m activation_sparse_decode_sigmoid_gb300.build")
    lib = ctypes.CDLL(path)
    P, I32, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32
    sig = {
        "pi_create": (st, [ctypes.POINTER(P), I32, P, I32, I32]),
        "pi_destroy": (st, [P]),
        "pi_set_stream": (st, [P, P]),
        "pi_load_layer": (st, [P, I32, ctypes.POINTER(pi_layer_desc), ctypes.POINTER(pi_layer_weights), P]),
        "pi_layer_counts": (st, [P, I32, P, I32, P]),
        "pi_perm_from_counts": (st, [P, I32, P]),
        "pi_predict": (st, [P, I32, P, I32, P, P]),
        "pi_sparse_ffn": (st, [P, I32, P, I32, P, P, P]),
        "pi_dense_ffn": (st, [P, I32, P, I32, P]),
        "pi_decode_step": (st, [P, P, I32]),
        "pi_decode_step_host": (st, [P, P, P, I32]),
        "pi_dense_step": (st, [P, P, I32]),
        "pi_set_trace": (st, [P, P, P, P, P]),
        "pi_sync_status": (st, [P]),
        "pi_last_error": (ctypes.c_char_p, [P]),
        "pi_grid_size": (I32, [P]),
        "pi_debug_set_wait_limit": (st, [P, ctypes.c_uint64]),
        "pi_debug_barrier_extra": (st, [P, I32]),
        "pi_debug_set_timeline": (st, [P, P, I32]),
        "pi_debug_set_tuning": (st, [P, I32, I32, I32, I32]),
        "pi_debug_copy_hidden": (st, [P, P, I32]),
        "pi_debug_set_mma_min_batch": (st, [P, I32]),
        "pi_sparse_ffn_noalloc": (st, [ctypes.POINTER(pi_ffn_rows), P, I32, P, P, P, P, P]),
        "pi_set_hot_prefix": (st, [P, I32, I32]),
        "pi_layerwise_min_batch": (st, [P, I32, P]),
        "pi_hot_prefix_crossover": (st, [P, I32, I32, I32, ctypes.c_double, ctypes.c_double, P]),
        "pi_choose_hot_prefix": (st, [P, I32, P, I32, I32, P]),
        "pi_load_layer_shard": (st, [P, I32, ctypes.POINTER(pi_layer_desc), ctypes.POINTER(pi_layer_weights), P,
                                     I32, I32]),
        "pi_layer_shard": (st, [P, I32, P, P]),
        "pi_layer_partial": (st, [P, I32, P, I32, P]),
        "pi_residual_add": (st, [P, P, P, I32]),
        "pi_linear_workspace": (st, [P, P, I32, P]),
        "pi_linear": (st, [P] * 9 + [ctypes.c_size_t]),
        "pi_linear_bwd": (st, [P] * 9 + [I32, P, ctypes.c_size_t]),
        "pi_gated_ffn_workspace": (st, [P, P, I32, P]),
        "pi_gated_ffn": (st, [P] * 7 + [ctypes.c_size_t]),
        "pi_gated_ffn_bwd": (st, [P] * 8 + [I32, P, ctypes.c_size_t]),
        "pi_norm_residual": (st, [P] * 8),
        "pi_norm_residual_bwd_workspace": (st, [P, P, P]),
        "pi_norm_residual_bwd": (st, [P] * 9 + [I32, P, ctypes.c_size_t]),
        "pi_mx_bytes": (st, [I32, I32, I32, P, P]),
        "pi_mx_quantize": (st, [P] * 4),
        "pi_mx_dequantize": (st, [P] * 4),
        "pi_mx_linear_workspace": (st, [P] * 3),
        "pi_mx_linear": (st, [P] * 8 + [ctypes.c_size_t]),
        "pi_mx_gated_ffn_workspace": (st, [P] * 3),
        "pi_mx_gated_ffn": (st, [P] * 6 + [ctypes.c_size_t]),
        "pi_norm_residual_mx": (st, [P, P, I32] + [P] * 6),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


_raw_stream = None


def _stream_ptr(device) -> int:
    """The handle of torch's current stream on `device`."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(device.index)


_torch = None


def _import_torch():
    """The module, imported on first use (an import statement in a call's path costs 0.3 us)."""
    global _torch
    import torch
    _torch = torch
    return torch


_CODES: dict = {}


def _codes() -> dict:
    """pi_dtype by torch type."""
    if not _CODES:
        import torch
        _CODES.update({torch.float16: PI_F16, torch.bfloat16: PI_BF16, torch.float32: PI_F32})
    return _CODES


# ---------------------------------------------------------------- same-named calls
def pi_create(device: int = 0, stream: int | None = None, max_layers: int = 1, max_batch: int = 1) -> int:
    lib = load_library()
    h = ctypes.c_void_p()
    rc = lib.pi_create(ctypes.byref(h), device, stream, max_layers, max_batch)
    if rc:
        raise PiError(rc, "pi_create failed")
    return h.value


def _check(ctx, rc, what):
    if rc:
        msg = load_library().pi_last_error(ctx)
        raise PiError(rc, f"{what}: {msg.decode() if msg else ''}")


def pi_destroy(ctx: int) -> None:
    _check(ctx, load_library().pi_destroy(ctx), "pi_destroy")


def pi_set_stream(ctx: int, stream: int | None) -> None:
    _check(ctx, load_library().pi_set_stream(ctx, stream), "pi_set_stream")


def pi_load_layer(ctx: int, layer: int, desc: pi_layer_desc, weights: pi_layer_weights, perm=None) -> None:
    perm_arr = None if perm is None else np.ascontiguousarray(perm, dtype=np.int32)
    rc = load_library().pi_load_layer(ctx, layer, ctypes.byref(desc), ctypes.byref(weights), _ptr(perm_arr))
    _check(ctx, rc, "pi_load_layer")


def pi_load_layer_shard(ctx: int, layer: int, desc: pi_layer_desc, weights: pi_layer_weights, perm, shard: int,
                        nshards: int) -> None:
    perm_arr = None if perm is None else np.ascontiguousarray(perm, dtype=np.int32)
    rc = load_library().pi_load_layer_shard(ctx, layer, ctypes.byref(desc), ctypes.byref(weights), _ptr(perm_arr),
                                            shard, nshards)
    _check(ctx, rc, "pi_load_layer_shard")


def pi_layer_shard(ctx: int, layer: int) -> tuple[int, int]:
    v = np.zeros(2, np.int32)
    _check(ctx, load_library().pi_layer_shard(ctx, layer, _ptr(v[0:1]), _ptr(v[1:2])), "pi_layer_shard")
    return int(v[0]), int(v[1])


def pi_layer_partial(ctx: int, layer: int, x, B: int, u) -> None:
    _check(ctx, load_library().pi_layer_partial(ctx, layer, _ptr(x), B, _ptr(u)), "pi_layer_partial")


def pi_residual_add(ctx: int, x, u, B: int) -> None:
    _check(ctx, load_library().pi_residual_add(ctx, _ptr(x), _ptr(u), B), "pi_residual_add")


def pi_layer_counts(ctx: int, layer: int, x_hat, T: int, counts) -> None:
    _check(ctx, load_library().pi_layer_counts(ctx, layer, _ptr(x_hat), T, _ptr(counts)), "pi_layer_counts")


def pi_perm_from_counts(counts) -> np.ndarray:
    c = np.ascontiguousarray(counts, dtype=np.int32)
    perm = np.empty(c.size, np.int32)
    rc = load_library().pi_perm_from_counts(_ptr(c), c.size, _ptr(perm))
    if rc:
        raise PiError(rc, "pi_perm_from_counts")
    return perm


def pi_set_hot_prefix(ctx: int, layer: int, hot: int) -> None:
    _check(ctx, load_library().pi_set_hot_prefix(ctx, layer, hot), "pi_set_hot_prefix")


def pi_hot_prefix_crossover(counts, T: int, B: int, pred_bytes: float, ffn_bytes: float) -> int:
    c = np.ascontiguousarray(counts, dtype=np.int32)
    hot = np.zeros(1, np.int32)
    rc = load_library().pi_hot_prefix_crossover(_ptr(c), c.size, T, B, pred_bytes, ffn_bytes, _ptr(hot))
    if rc:
        raise PiError(rc, "pi_hot_prefix_crossover")
    return int(hot[0])


def pi_choose_hot_prefix(ctx: int, layer: int, counts, T: int, B: int) -> int:
    c = np.ascontiguousarray(counts, dtype=np.int32)
    hot = np.zeros(1, np.int32)
    _check(ctx, load_library().pi_choose_hot_prefix(ctx, layer, _ptr(c), T, B, _ptr(hot)), "pi_choose_hot_prefix")
    return int(hot[0])


def pi_predict(ctx: int, layer: int, x_hat, B: int, idx, count) -> None:
    _check(ctx, load_library().pi_predict(ctx, layer, _ptr(x_hat), B, _ptr(idx), _ptr(count)), "pi_predict")


def pi_sparse_ffn(ctx: int, layer: int, x_hat, B: int, idx, count, y) -> None:
    rc = load_library().pi_sparse_ffn(ctx, layer, _ptr(x_hat), B, _ptr(idx), _ptr(count), _ptr(y))
    _check(ctx, rc, "pi_sparse_ffn")


def pi_sparse_ffn_noalloc(rows: pi_ffn_rows, x_hat, B: int, idx, count, y, dev_status=None,
                          stream: int | None = None) -> int:
    """Context-free sparse FFN that allocates nothing (for callers that may
    not call cudaMalloc); scratch lives in a fixed per-GPU array inside the
    library.  Returns the status instead of raising.  `stream` defaults to
    torch's current stream."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    return load_library().pi_sparse_ffn_noalloc(ctypes.byref(rows), _ptr(x_hat), B, _ptr(idx), _ptr(count),
                                                 _ptr(y), _ptr(dev_status), stream)


def pi_dense_ffn(ctx: int, layer: int, x_hat, B: int, y) -> None:
    _check(ctx, load_library().pi_dense_ffn(ctx, layer, _ptr(x_hat), B, _ptr(y)), "pi_dense_ffn")


def pi_decode_step(ctx: int, x, B: int) -> None:
    _check(ctx, load_library().pi_decode_step(ctx, _ptr(x), B), "pi_decode_step")


def pi_decode_step_host(ctx: int, x_in, x_out, B: int) -> None:
    """x_in / x_out: host fp32 [B][d] (numpy arrays or CPU tensors, ideally pinned)."""
    _check(ctx, load_library().pi_decode_step_host(ctx, _ptr(x_in), _ptr(x_out), B), "pi_decode_step_host")


def pi_dense_step(ctx: int, x, B: int) -> None:
    _check(ctx, load_library().pi_dense_step(ctx, _ptr(x), B), "pi_dense_step")


def pi_set_trace(ctx: int, x_trace=None, xhat_trace=None, idx_trace=None, count_trace=None) -> None:
    rc = load_library().pi_set_trace(ctx, _ptr(x_trace), _ptr(xhat_trace), _ptr(idx_trace), _ptr(count_trace))
    _check(ctx, rc, "pi_set_trace")


def pi_sync_status(ctx: int) -> int:
    """Returns the status (0 = OK) instead of raising, so callers can test it."""
    return load_library().pi_sync_status(ctx)


def pi_last_error(ctx: int) -> str:
    m = load_library().pi_last_error(ctx)
    return m.decode() if m else ""


def pi_grid_size(ctx: int) -> int:
    return load_library().pi_grid_size(ctx)


def pi_debug_set_wait_limit(ctx: int, ns: int) -> None:
    _check(ctx, load_library().pi_debug_set_wait_limit(ctx, ns), "pi_debug_set_wait_limit")


def pi_debug_set_timeline(ctx: int, stamps=None, per_cta: int = 0) -> None:
    _check(ctx, load_library().pi_debug_set_timeline(ctx, _ptr(stamps), per_cta), "pi_debug_set_timeline")


def pi_debug_set_tuning(ctx: int, prefetch: int, prefetch_ns: int, lookahead: int, rows_ahead: int = 0) -> None:
    rc = load_library().pi_debug_set_tuning(ctx, prefetch, prefetch_ns, lookahead, rows_ahead)
    _check(ctx, rc, "pi_debug_set_tuning")


def pi_debug_copy_hidden(ctx: int, dst, count: int) -> None:
    _check(ctx, load_library().pi_debug_copy_hidden(ctx, _ptr(dst), count), "pi_debug_copy_hidden")


def pi_debug_set_mma_min_batch(ctx: int, min_batch: int) -> None:
    _check(ctx, load_library().pi_debug_set_mma_min_batch(ctx, min_batch), "pi_debug_set_mma_min_batch")


def pi_layerwise_min_batch(ctx: int, layer: int) -> int:
    mb = np.zeros(1, np.int32)
    _check(ctx, load_library().pi_layerwise_min_batch(ctx, layer, _ptr(mb)), "pi_layerwise_min_batch")
    return int(mb[0])


def pi_debug_barrier_extra(ctx: int, extra: int) -> None:
    _check(ctx, load_library().pi_debug_barrier_extra(ctx, extra), "pi_debug_barrier_extra")


def _ref(struct) -> int | None:
    return None if struct is None else ctypes.addressof(struct)


def pi_linear_workspace(ctx: int, desc, backward: bool) -> int:
    n = ctypes.c_size_t()
    _check(ctx, load_library().pi_linear_workspace(ctx, _ref(desc), int(backward), ctypes.addressof(n)),
           "pi_linear_workspace")
    return n.value


def pi_linear(ctx: int, desc, x, w, b, residual, z, y, ws, ws_bytes: int) -> None:
    rc = load_library().pi_linear(ctx, _ref(desc), _ptr(x), _ptr(w), _ptr(b), _ptr(residual), _ptr(z), _ptr(y), _ptr(ws),
                                  ws_bytes)
    _check(ctx, rc, "pi_linear")


def pi_linear_bwd(ctx: int, desc, dy, x, w, z, dx, dw, db, accumulate: bool, ws, ws_bytes: int) -> None:
    rc = load_library().pi_linear_bwd(ctx, _ref(desc), _ptr(dy), _ptr(x), _ptr(w), _ptr(z), _ptr(dx), _ptr(dw), _ptr(db),
                                      int(accumulate), _ptr(ws), ws_bytes)
    _check(ctx, rc, "pi_linear_bwd")


def pi_gated_ffn_workspace(ctx: int, desc, backward: bool) -> int:
    n = ctypes.c_size_t()
    _check(ctx, load_library().pi_gated_ffn_workspace(ctx, _ref(desc), int(backward), ctypes.addressof(n)),
           "pi_gated_ffn_workspace")
    return n.value


def pi_gated_ffn(ctx: int, desc, weights, x, save, y, ws, ws_bytes: int) -> None:
    rc = load_library().pi_gated_ffn(ctx, _ref(desc), _ref(weights), _ptr(x), _ref(save), _ptr(y), _ptr(ws), ws_bytes)
    _check(ctx, rc, "pi_gated_ffn")


def pi_gated_ffn_bwd(ctx: int, desc, weights, x, dy, save, dx, grads, accumulate: bool, ws, ws_bytes: int) -> None:
    rc = load_library().pi_gated_ffn_bwd(ctx, _ref(desc), _ref(weights), _ptr(x), _ptr(dy), _ref(save), _ptr(dx),
                                         _ref(grads), int(accumulate), _ptr(ws), ws_bytes)
    _check(ctx, rc, "pi_gated_ffn_bwd")


def pi_norm_residual(ctx: int, desc, params, x, y, gate, x_out, h) -> None:
    rc = load_library().pi_norm_residual(ctx, _ref(desc), _ref(params), _ptr(x), _ptr(y), _ptr(gate), _ptr(x_out),
                                         _ptr(h))
    _check(ctx, rc, "pi_norm_residual")


def pi_norm_residual_bwd_workspace(ctx: int, desc) -> int:
    n = ctypes.c_size_t()
    _check(ctx, load_library().pi_norm_residual_bwd_workspace(ctx, _ref(desc), ctypes.addressof(n)),
           "pi_norm_residual_bwd_workspace")
    return n.value


def pi_norm_residual_bwd(ctx: int, desc, params, dx_out, dh, x_out, y, gate, grads, accumulate: bool, ws,
                         ws_bytes: int) -> None:
    rc = load_library().pi_norm_residual_bwd(ctx, _ref(desc), _ref(params), _ptr(dx_out), _ptr(dh), _ptr(x_out), _ptr(y),
                                             _ptr(gate), _ref(grads), int(accumulate), _ptr(ws), ws_bytes)
    _check(ctx, rc, "pi_norm_residual_bwd")


def pi_mx_bytes(rows: int, cols: int, kind: int) -> tuple[int, int]:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    rc = load_library().pi_mx_bytes(rows, cols, kind, ctypes.addressof(a), ctypes.addressof(b))
    if rc:
        raise PiError(rc, f"pi_mx_bytes: {rows} rows, {cols} columns, kind {kind}")
    return a.value, b.value


def pi_mx_quantize(ctx: int, desc, x, q) -> None:
    _check(ctx, load_library().pi_mx_quantize(ctx, _ref(desc), _ptr(x), _ref(q)), "pi_mx_quantize")


def pi_mx_dequantize(ctx: int, desc, q, y) -> None:
    _check(ctx, load_library().pi_mx_dequantize(ctx, _ref(desc), _ref(q), _ptr(y)), "pi_mx_dequantize")


def pi_mx_linear_workspace(ctx: int, desc) -> int:
    n = ctypes.c_size_t()
    _check(ctx, load_library().pi_mx_linear_workspace(ctx, _ref(desc), ctypes.addressof(n)), "pi_mx_linear_workspace")
    return n.value


def pi_mx_linear(ctx: int, desc, x, w, b, residual, y, ws, ws_bytes: int) -> None:
    rc = load_library().pi_mx_linear(ctx, _ref(desc), _ref(x), _ref(w), _ptr(b), _ptr(residual), _ptr(y), _ptr(ws), ws_bytes)
    _check(ctx, rc, "pi_mx_linear")


def pi_mx_gated_ffn_workspace(ctx: int, desc) -> int:
    n = ctypes.c_size_t()
    _check(ctx, load_library().pi_mx_gated_ffn_workspace(ctx, _ref(desc), ctypes.addressof(n)), "pi_mx_gated_ffn_workspace")
    return n.value


def pi_mx_gated_ffn(ctx: int, desc, weights, x, y, ws, ws_bytes: int) -> None:
    rc = load_library().pi_mx_gated_ffn(ctx, _ref(desc), _ref(weights), _ref(x), _ptr(y), _ptr(ws), ws_bytes)
    _check(ctx, rc, "pi_mx_gated_ffn")


def pi_norm_residual_mx(ctx: int, desc, kind: int, params, x, y, gate, x_out, h) -> None:
    rc = load_library().pi_norm_residual_mx(ctx, _ref(desc), kind, _ref(params), _ptr(x), _ptr(y), _ptr(gate), _ptr(x_out),
                                            _ref(h))
    _check(ctx, rc, "pi_norm_residual_mx")


class MxMatrix:
    """A microscaled matrix [rows][cols] of kind PI_MX8 or PI_MX4: `codes`
    uint8 [rows][bytes of a padded row], `scales` uint8 [row tiles][column
    tiles][32][4][4] (include/pi.h has the layout).  ``Context.mx_quantize``
    and ``Context.mx_empty`` make them; another program's are wrapped as they are."""

    __slots__ = ("codes", "scales", "cols", "kind")

    def __init__(self, codes, scales, cols: int, kind: int):
        if kind != PI_MX8 and kind != PI_MX4:
            raise PiError(PI_ERR_ARG, f"kind {kind} is not PI_MX8 or PI_MX4")
        self.codes, self.scales, self.cols, self.kind = codes, scales, cols, kind

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def shape(self) -> tuple[int, int]:
        return self.codes.shape[0], self.cols


# ---------------------------------------------------------------- convenience wrapper
class Context:
    """Owns a pi_ctx; every call runs on torch's current stream of `device`."""

    _plans: dict = {}  # (see _plan; a context's own is set when it is created)

    def __init__(self, device: int = 0, max_layers: int = 1, max_batch: int = 1):
        import torch
        self.device = device
        self.torch_device = torch.device("cuda", device)
        self.max_layers, self.max_batch = max_layers, max_batch
        self._plans = {}
        self.handle = pi_create(device, _stream_ptr(self.torch_device), max_layers, max_batch)
        self.descs: dict[int, pi_layer_desc] = {}
        self.hot: dict[int, int] = {}  # each layer's always-active prefix

    def close(self):
        if self.handle:
            pi_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _s(self):
        rc = _lib.pi_set_stream(self.handle, _stream_ptr(self.torch_device))
        if rc:
            _check(self.handle, rc, "pi_set_stream")

    @property
    def grid(self) -> int:
        return pi_grid_size(self.handle)

    # -- loading
    def load_layer(self, layer: int, lw: dict, perm=None) -> None:
        """Load a layer dict as drawn by ``workload.make_layer`` (numpy, host)
        or ``workload.make_layer_device`` (torch, device)."""
        desc, w, keep = self._weights(lw)
        self._s()
        pi_load_layer(self.handle, layer, desc, w, perm)
        self.descs[layer] = desc
        self.hot[layer] = 0
        del keep

    def _weights(self, lw: dict):
        """(descriptor, weight pointers, the buffers they point into) of a layer dict."""
        desc = pi_layer_desc(lw["d"], lw["n"], lw["r"], lw["act"], lw["w_dtype"], lw["act_dtype"])
        keys = ("w_up", "w_gate", "b", "w_down", "b_down", "p_w1", "p_b1", "p_w2", "p_b2")
        vals = [lw.get(k) for k in keys]
        on_dev = any(v is not None and not isinstance(v, np.ndarray) for v in vals)
        keep = []
        ptrs = []
        for v in vals:
            if v is None:
                ptrs.append(None)
                continue
            if on_dev and isinstance(v, np.ndarray):
                import torch
                v = torch.from_numpy(np.ascontiguousarray(v).view(np.int16) if v.dtype == np.uint16 else
                                     np.ascontiguousarray(v)).to(self.torch_device)
            elif isinstance(v, np.ndarray):
                v = np.ascontiguousarray(v)
            else:
                v = v.contiguous()
            keep.append(v)
            ptrs.append(_ptr(v))
        w = pi_layer_weights(*ptrs, 1 if on_dev else 0)
        return desc, w, keep

    def load_layer_shard(self, layer: int, lw: dict, shard: int, nshards: int, perm=None) -> None:
        """Load shard `shard` of `nshards` of a layer dict (its physical
        neurons shard, shard + nshards, ...)."""
        desc, w, keep = self._weights(lw)
        self._s()
        pi_load_layer_shard(self.handle, layer, desc, w, perm, shard, nshards)
        n = lw["n"]
        desc.d_ffn = (n - shard + nshards - 1) // nshards
        self.descs[layer] = desc
        self.hot[layer] = 0
        del keep

    def layer_partial(self, layer: int, x, u=None):
        """The layer's fp32 update of the residual x ([B][d]), not added."""
        import torch
        if u is None:
            u = torch.empty_like(x)
        self._s()
        pi_layer_partial(self.handle, layer, x, x.shape[0], u)
        return u

    def residual_add(self, x, u) -> None:
        self._s()
        pi_residual_add(self.handle, x, u, x.shape[0])

    def layer_counts(self, layer: int, x_hat):
        import torch
        n = self.descs[layer].d_ffn
        counts = torch.zeros(n, dtype=torch.int32, device=self.torch_device)
        self._s()
        pi_layer_counts(self.handle, layer, x_hat, x_hat.shape[0], counts)
        return counts

    def set_hot_prefix(self, layer: int, hot: int) -> None:
        self._s()
        pi_set_hot_prefix(self.handle, layer, hot)
        self.hot[layer] = hot

    def choose_hot_prefix(self, layer: int, counts, T: int, B: int) -> int:
        """Crossover prefix length from calibration counts (host or device, physical order)."""
        if not isinstance(counts, np.ndarray):
            counts = counts.cpu().numpy()
        return pi_choose_hot_prefix(self.handle, layer, counts, T, B)

    # -- hot path
    def predict(self, layer: int, x_hat, idx=None, count=None):
        import torch
        n = self.descs[layer].d_ffn
        if idx is None:
            idx = torch.empty(n, dtype=torch.int32, device=self.torch_device)
        if count is None:
            count = torch.empty(1, dtype=torch.int32, device=self.torch_device)
        self._s()
        pi_predict(self.handle, layer, x_hat, x_hat.shape[0], idx, count)
        return idx, count

    def _y(self, layer, B, y):
        import torch
        if y is None:
            d = self.descs[layer]
            dt = torch.bfloat16 if d.act_dtype == PI_BF16 else torch.float16
            y = torch.empty((B, d.d_model), dtype=dt, device=self.torch_device)
        return y

    def sparse_ffn(self, layer: int, x_hat, idx, count, y=None):
        y = self._y(layer, x_hat.shape[0], y)
        self._s()
        pi_sparse_ffn(self.handle, layer, x_hat, x_hat.shape[0], idx, count, y)
        return y

    def dense_ffn(self, layer: int, x_hat, y=None):
        y = self._y(layer, x_hat.shape[0], y)
        self._s()
        pi_dense_ffn(self.handle, layer, x_hat, x_hat.shape[0], y)
        return y

    def decode_step(self, x) -> None:
        self._s()
        pi_decode_step(self.handle, x, x.shape[0])

    def decode_step_host(self, x_in, x_out) -> None:
        self._s()
        pi_decode_step_host(self.handle, x_in, x_out, x_in.shape[0])

    def dense_step(self, x) -> None:
        self._s()
        pi_dense_step(self.handle, x, x.shape[0])

    # -- block operators: long prompts and training (tensors of torch's float16, bfloat16 and float32)
    # Calls of few tokens take less time on the GPU than here, so the checks
    # are written for the good case: _at() compares what a tensor is with what
    # is expected and leaves the reason for a refusal to _refuse(); a call's
    # desc and workspace size are kept by its sizes, types and strides.
    def _at(self, name, t, shape, dtype):
        """(address, row stride) of a matrix or vector, 0 for packed rows (the
        stride of a single row says nothing); (0, 0) of None."""
        if t is None:
            return 0, 0
        if t.dtype != dtype or t.shape != shape or t.device != self.torch_device:
            self._refuse(name, t, shape, dtype)
        if t.is_contiguous():
            return t.data_ptr(), 0
        st = t.stride()
        if (st[-1] != 1 and shape[-1] > 1) or (len(shape) == 2 and shape[0] > 1 and st[0] < shape[1]):
            self._refuse(name, t, shape, dtype)
        return t.data_ptr(), st[0] if len(shape) == 2 and shape[0] > 1 else 0

    def _refuse(self, name, t, shape, dtype):
        if t.device != self.torch_device:
            raise PiError(PI_ERR_ARG, f"{name} is on {t.device}, the context on {self.torch_device}")
        if t.dtype != dtype:
            raise PiError(PI_ERR_ARG, f"{name} is {t.dtype}, expected {dtype}")
        if tuple(t.shape) != tuple(shape):
            raise PiError(PI_ERR_SHAPE, f"{name} is {list(t.shape)}, expected {list(shape)}")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise PiError(PI_ERR_ARG, f"{name}: a row's elements are not consecutive")
        raise PiError(PI_ERR_SHAPE, f"{name}: rows overlap (stride {t.stride(0)})")

    @staticmethod
    def _dims(name, t):
        if t.dim() != 2:
            raise PiError(PI_ERR_SHAPE, f"{name} has {t.dim()} dimensions, expected 2")
        return t.shape

    @staticmethod
    def _code(dtype) -> int:
        code = (_CODES or _codes()).get(dtype)
        if code is None:
            raise PiError(PI_ERR_ARG, f"type {dtype} is not float16, bfloat16 or float32")
        return code

    @staticmethod
    def _code16(dtype) -> int:
        code = (_CODES or _codes()).get(dtype)
        if code is None or code == PI_F32:
            raise PiError(PI_ERR_ARG, f"dtype {dtype} is not float16 or bfloat16")
        return code

    def _plan(self, kind, fields, query, *more):
        """(desc, workspace bytes) of a call, by the desc's fields."""
        plans = self._plans
        key = (kind, fields, query, more)
        got = plans.get(key)
        if got is None:
            desc = kind(*fields)
            got = plans[key] = desc, (query(self.handle, desc, *more) if query else 0)
            if len(plans) > 4096:  # (a program of ever new lengths)
                plans.clear()
        return got

    def _new(self, shape, dtype):
        return (_torch or _import_torch()).empty(shape, dtype=dtype, device=self.torch_device)

    def _ws(self, n: int):
        """Workspace of n bytes and its address."""
        if not n:
            return None, 0
        torch = _torch or _import_torch()
        t = torch.empty(n, dtype=torch.uint8, device=self.torch_device)
        return t, t.data_ptr()

    def _grad_buffers(self, given: dict, shapes: dict, dtype):
        """Checks gradient buffers: packed, one type; returns that type."""
        kind = None
        for k, t in given.items():
            if t is None:
                continue
            if kind is None:
                kind = t.dtype
                if kind != dtype and self._code(kind) != PI_F32:
                    raise PiError(PI_ERR_ARG, f"gradient of {k} is {kind}, expected {dtype} or float32")
            elif t.dtype != kind:
                raise PiError(PI_ERR_ARG, f"gradient of {k} is {t.dtype}, another's {kind}")
            self._at("gradient of " + k, t, shapes[k], kind)
            if not t.is_contiguous():
                raise PiError(PI_ERR_ARG, f"gradient of {k} is not packed")
        return kind or dtype

    def linear(self, x, w, b=None, *, fn=PI_FN_NONE, scale=1.0, residual=None, z=None, y=None):
        """y = residual + scale * fn(x W^T + b).  y is x's type, or the
        residual's (float32 residual stream); z, if given, receives
        x W^T + b for the backward pass."""
        dt = x.dtype
        code = self._code16(dt)
        T, K = self._dims("x", x)
        N = self._dims("w", w)[0]
        if y is None:
            y = self._new((T, N), dt if residual is None else residual.dtype)
        out = self._code(y.dtype)
        px, ldx = self._at("x", x, (T, K), dt)
        pw, ldw = self._at("w", w, (N, K), dt)
        pb, _ = self._at("b", b, (N,), dt)
        pr, ldr = self._at("residual", residual, (T, N), y.dtype)
        pz, ldz = self._at("z", z, (T, N), dt)
        py, ldy = self._at("y", y, (T, N), y.dtype)
        desc, n = self._plan(pi_linear_desc, (T, K, N, code, out, code, fn, scale, (px | pw) & 15 != 0, ldx, ldw, ldz, ldr,
                                              ldy, 0, 0), pi_linear_workspace, False)
        ws, pws = self._ws(n)
        self._s()
        rc = _lib.pi_linear(self.handle, ctypes.addressof(desc), px, pw, pb, pr, pz, py, pws, n)
        if rc:
            _check(self.handle, rc, "pi_linear")
        return y

    def linear_bwd(self, dy, x, w, z=None, *, fn=PI_FN_NONE, scale=1.0, need=(True, True, True), dx=None, dw=None,
                   db=None, accumulate=False):
        """(dx, dw, db) of ``linear`` for the gradient dy of y (the residual's
        is dy itself).  need: which of them; buffers may be given, dw and db
        in x's type or float32, and are added to with `accumulate`."""
        dt = x.dtype
        code = self._code16(dt)
        T, K = self._dims("x", x)
        N = self._dims("w", w)[0]
        if accumulate and any(n and g is None for n, g in zip(need[1:], (dw, db))):
            raise PiError(PI_ERR_ARG, "accumulate needs the buffers that it adds to")
        gdt = dt if not (need[1] or need[2]) else next((t.dtype for t in (dw, db) if t is not None), dt)
        grad = self._code(gdt)
        dx = (self._new((T, K), dt) if dx is None else dx) if need[0] else None
        dw = (self._new((N, K), gdt) if dw is None else dw) if need[1] else None
        db = (self._new((N,), gdt) if db is None else db) if need[2] else None
        pdy, ldy = self._at("dy", dy, (T, N), dy.dtype)
        px, ldx = self._at("x", x, (T, K), dt)
        pw, ldw = self._at("w", w, (N, K), dt)
        pz, ldz = self._at("z", z, (T, N), dt)
        pdx, lddx = self._at("dx", dx, (T, K), dt)
        pdw, lddw = self._at("dw", dw, (N, K), gdt)
        pdb, _ = self._at("db", db, (N,), gdt)
        desc, n = self._plan(pi_linear_desc, (T, K, N, code, self._code(dy.dtype), grad, fn, scale,
                                              (pdy | px | pw) & 15 != 0, ldx, ldw, ldz, 0, ldy, lddx, lddw),
                             pi_linear_workspace, True)
        ws, pws = self._ws(n)
        self._s()
        rc = _lib.pi_linear_bwd(self.handle, ctypes.addressof(desc), pdy, px, pw, pz, pdx, pdw, pdb,
                                          int(accumulate), pws, n)
        if rc:
            _check(self.handle, rc, "pi_linear_bwd")
        return dx, dw, db

    def gated_ffn_save(self, x, w_gate, w_up):
        """Buffers (g, u, a) for ``gated_ffn`` to leave for its backward pass,
        [T][n] with rows that start on 16-byte boundaries (g None if not gated)."""
        torch = _torch or _import_torch()
        T, n = x.shape[0], w_up.shape[0]
        new = lambda: torch.empty_strided((T, n), ((n + 7) // 8 * 8, 1), dtype=x.dtype, device=x.device)
        return (new() if w_gate is not None else None), new(), new()

    def gated_ffn(self, x, w_gate, w_up, w_down, b_gate=None, b_up=None, b_down=None, *, fn=PI_FN_RELU, save=None,
                  y=None):
        """y = (fn(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd, weights in the
        model's layout; w_gate None: y = fn(x Wu^T + bu) Wd^T + bd.  save
        (``gated_ffn_save``) keeps g, u and a for the backward pass."""
        dt = x.dtype
        code = self._code16(dt)
        T, d = self._dims("x", x)
        n = self._dims("w_up", w_up)[0]
        if y is None:
            y = self._new((T, d), dt)
        g, u, a = save if save is not None else (None, None, None)
        px, ldx = self._at("x", x, (T, d), dt)
        pwg, ldwg = self._at("w_gate", w_gate, (n, d), dt)
        pwu, ldwu = self._at("w_up", w_up, (n, d), dt)
        pwd, ldwd = self._at("w_down", w_down, (d, n), dt)
        pg, ldg = self._at("g", g, (T, n), dt)
        pu, ldu = self._at("u", u, (T, n), dt)
        pa, lda = self._at("a", a, (T, n), dt)
        py, ldy = self._at("y", y, (T, d), dt)
        pbg, pbu = self._at("b_gate", b_gate, (n,), dt)[0], self._at("b_up", b_up, (n,), dt)[0]
        pbd = self._at("b_down", b_down, (d,), dt)[0]
        desc, nb = self._plan(pi_gated_ffn_desc, (T, d, n, code, code, fn, w_gate is not None,
                                                  (px | pwg | pwu | pwd | pa) & 15 != 0, ldx, ldy, ldwg, ldwu, ldwd, ldg,
                                                  ldu, lda), pi_gated_ffn_workspace, False)
        wts, sv = pi_gated_ffn_weights(pwg, pwu, pwd, pbg, pbu, pbd), pi_gated_ffn_save(pg, pu, pa)
        ws, pws = self._ws(nb)
        self._s()
        rc = _lib.pi_gated_ffn(self.handle, ctypes.addressof(desc), ctypes.addressof(wts), px,
                                         ctypes.addressof(sv), py, pws, nb)
        if rc:
            _check(self.handle, rc, "pi_gated_ffn")
        return y

    def gated_ffn_bwd(self, dy, x, w_gate, w_up, w_down, save, *, fn=PI_FN_RELU, need_dx=True, weight_grads=True,
                      bias_grads=True, grads=None, accumulate=False):
        """Gradients of ``gated_ffn`` for the gradient dy of y, as a dict with
        keys dx, w_gate, w_up, w_down, b_gate, b_up, b_down (None: not
        wanted).  grads: the parameter gradients' buffers by the same keys,
        packed, in x's type or float32 (all alike), used instead of new ones
        and added to with `accumulate`; then only the given ones are computed."""
        dt = x.dtype
        code = self._code16(dt)
        g, u, a = save
        T, d = self._dims("x", x)
        n, gated = self._dims("w_up", w_up)[0], w_gate is not None
        if grads is None:
            if accumulate:
                raise PiError(PI_ERR_ARG, "accumulate needs the buffers that it adds to")
            new, w, b = self._new, weight_grads, bias_grads
            out = {"w_gate": new((n, d), dt) if w and gated else None, "w_up": new((n, d), dt) if w else None,
                   "w_down": new((d, n), dt) if w else None, "b_gate": new((n,), dt) if b and gated else None,
                   "b_up": new((n,), dt) if b else None, "b_down": new((d,), dt) if b else None}
            gdt = dt
        else:
            shapes = {"w_gate": (n, d), "w_up": (n, d), "w_down": (d, n), "b_gate": (n,), "b_up": (n,), "b_down": (d,)}
            out = {k: grads.get(k) for k in shapes}
            gdt = self._grad_buffers(out, shapes, dt)
        pdy, ldy = self._at("dy", dy, (T, d), dt)
        px, ldx = self._at("x", x, (T, d), dt)
        dx = None
        if need_dx:  # (x and dx share their stride)
            dx = self._new((T, d), dt) if ldx in (0, d) else self._new((T, ldx), dt)[:, :d]
        pwg, ldwg = self._at("w_gate", w_gate, (n, d), dt)
        pwu, ldwu = self._at("w_up", w_up, (n, d), dt)
        pwd, ldwd = self._at("w_down", w_down, (d, n), dt)
        pg, ldg = self._at("g", g, (T, n), dt)
        pu, ldu = self._at("u", u, (T, n), dt)
        pa, lda = self._at("a", a, (T, n), dt)
        desc, nb = self._plan(pi_gated_ffn_desc, (T, d, n, code, self._code(gdt), fn, gated,
                                                  (pdy | px | pwg | pwu | pwd | pa) & 15 != 0, ldx, ldy, ldwg, ldwu, ldwd,
                                                  ldg, ldu, lda), pi_gated_ffn_workspace, True)
        wts, sv = pi_gated_ffn_weights(pwg, pwu, pwd, 0, 0, 0), pi_gated_ffn_save(pg, pu, pa)
        gr = pi_gated_ffn_grads(*(_ptr(v) for v in out.values()))
        ws, pws = self._ws(nb)
        self._s()
        rc = _lib.pi_gated_ffn_bwd(self.handle, ctypes.addressof(desc), ctypes.addressof(wts), px, pdy,
                                             ctypes.addressof(sv), _ptr(dx), ctypes.addressof(gr), int(accumulate),
                                             pws, nb)
        if rc:
            _check(self.handle, rc, "pi_gated_ffn_bwd")
        return {"dx": dx, **out}

    def norm_residual(self, x, y=None, gate=None, *, pre=PI_NORM_RMS, post=PI_NORM_NONE, w_pre=None, b_pre=None,
                      w_post=None, b_post=None, res_scale=1.0, branch_scale=1.0, gate_rows=0, eps=1e-5, dtype=None,
                      x_out=None, h=None):
        """(x', h): x' = res_scale * x + branch_scale * gate * norm_post(y),
        h = norm_pre(x') in y's type (`dtype` without a y).  gate [rows][d]:
        token t uses row t // gate_rows, 0 = one row for all.  x_out may be x."""
        xdt = x.dtype
        xcode = self._code(xdt)
        if y is not None:
            dtype = y.dtype
        elif dtype is None:
            import torch
            dtype = torch.bfloat16 if xcode == PI_F32 else xdt
        code = self._code16(dtype)
        T, d = self._dims("x", x)
        if x_out is None:
            x_out = self._new((T, d), xdt)
        if h is None and pre != PI_NORM_NONE:
            h = self._new((T, d), dtype)
        px, ldx = self._at("x", x, (T, d), dtype if xcode != PI_F32 else xdt)
        py, ldy = self._at("y", y, (T, d), dtype)
        pg, ldg = self._at("gate", gate, (1 if gate_rows == 0 else -(-T // max(gate_rows, 1)), d), dtype)
        po, ldo = self._at("x_out", x_out, (T, d), xdt)
        ph, ldh = self._at("h", h, (T, d), dtype)
        par = pi_norm_residual_params(self._at("w_pre", w_pre, (d,), dtype)[0], self._at("b_pre", b_pre, (d,), dtype)[0],
                                      self._at("w_post", w_post, (d,), dtype)[0], self._at("b_post", b_post, (d,), dtype)[0])
        desc, _ = self._plan(pi_norm_residual_desc, (T, d, xcode, code, code, pre, post, gate_rows, res_scale, branch_scale,
                                                     eps, ldx, ldo, ldy, ldh, ldg), None)
        self._s()
        rc = _lib.pi_norm_residual(self.handle, ctypes.addressof(desc), ctypes.addressof(par), px, py, pg, po, ph)
        if rc:
            _check(self.handle, rc, "pi_norm_residual")
        return x_out, h

    def norm_residual_bwd(self, dx_out, dh, x_out, y=None, gate=None, *, pre=PI_NORM_RMS, post=PI_NORM_NONE, w_pre=None,
                          b_pre=None, w_post=None, b_post=None, res_scale=1.0, branch_scale=1.0, gate_rows=0, eps=1e-5,
                          grads=None, accumulate=False):
        """Gradients of ``norm_residual`` for the gradients dx_out of x' (None:
        0) and dh of h, as a dict with keys dx, dy, gate, w_pre, b_pre,
        w_post, b_post; a parameter that was not given, or that no norm or
        block used, has none.  grads:
        buffers for gate and the parameters, packed, in h's type or float32
        (all alike), used instead of new ones and added to with `accumulate`."""
        xdt = x_out.dtype
        xcode = self._code(xdt)
        if dh is None and y is None:
            raise PiError(PI_ERR_ARG, "neither dh nor y given")
        dtype = (dh if dh is not None else y).dtype
        code = self._code16(dtype)
        T, d = self._dims("x_out", x_out)
        rows = 1 if gate_rows == 0 else -(-T // max(gate_rows, 1))
        given = {"gate": gate, "w_pre": w_pre, "b_pre": b_pre, "w_post": w_post, "b_post": b_post}
        if grads is None:
            if accumulate:
                raise PiError(PI_ERR_ARG, "accumulate needs the buffers that it adds to")
            used = {"gate": y is not None, "pre": pre != PI_NORM_NONE, "post": y is not None and post != PI_NORM_NONE}
            out = {k: self._new(v.shape, dtype) if v is not None and used[k[2:] if k != "gate" else k] else None
                   for k, v in given.items()}
            gdt = dtype
        else:
            out = {k: grads.get(k) for k in given}
            gdt = self._grad_buffers(out, {k: (rows, d) if k == "gate" else (d,) for k in given}, dtype)
        if xcode != PI_F32 and xdt != dtype:
            raise PiError(PI_ERR_ARG, f"x_out is {xdt}, expected {dtype} or float32")
        px, ldxo = self._at("x_out", x_out, (T, d), xdt)
        pdxo, lddxo = self._at("dx_out", dx_out, (T, d), xdt)
        pdh, ldh = self._at("dh", dh, (T, d), dtype)
        py, ldy = self._at("y", y, (T, d), dtype)
        pg, ldg = self._at("gate", gate, (rows, d), dtype)
        par = pi_norm_residual_params(self._at("w_pre", w_pre, (d,), dtype)[0], self._at("b_pre", b_pre, (d,), dtype)[0],
                                      self._at("w_post", w_post, (d,), dtype)[0], self._at("b_post", b_post, (d,), dtype)[0])
        dx = self._new((T, d), xdt)
        # (y and dy share their stride)
        dy = None if y is None else self._new((T, d), dtype) if ldy in (0, d) else self._new((T, ldy), dtype)[:, :d]
        desc, n = self._plan(pi_norm_residual_desc, (T, d, xcode, code, self._code(gdt), pre, post, gate_rows, res_scale,
                                                     branch_scale, eps, 0, ldxo, ldy, ldh, ldg, lddxo or d),
                             pi_norm_residual_bwd_workspace)
        gr = pi_norm_residual_grads(dx.data_ptr(), _ptr(dy), *(_ptr(v) for v in out.values()))
        ws, pws = self._ws(n)
        self._s()
        rc = _lib.pi_norm_residual_bwd(self.handle, ctypes.addressof(desc), ctypes.addressof(par), pdxo, pdh, px,
                                                 py, pg, ctypes.addressof(gr), int(accumulate), pws, n)
        if rc:
            _check(self.handle, rc, "pi_norm_residual_bwd")
        return {"dx": dx, "dy": dy, **out}

    # -- microscaled matrices: the same block's forward side in 8 and 4 bits
    def _mx(self, name, q, rows, cols, kind=None):
        """(address of the codes, of the scales, row stride in bytes: 0 packed)"""
        if q is None:
            return 0, 0, 0
        if not isinstance(q, MxMatrix):
            self._mx_dims(name, q)
        if kind is not None and q.kind != kind:
            raise PiError(PI_ERR_ARG, f"{name} is of kind {q.kind}, expected {kind}")
        if q.cols != cols:
            raise PiError(PI_ERR_SHAPE, f"{name} has {q.cols} columns, expected {cols}")
        u8 = (_torch or _import_torch()).uint8
        B = (cols + 127) // 128
        codes, ld = self._at(name + ".codes", q.codes, (rows, B * (128 if q.kind == PI_MX8 else 64)), u8)
        s, want = q.scales, ((rows + 127) // 128, B, 32, 4, 4)
        if s.dtype != u8 or s.device != self.torch_device or s.shape != want:
            self._refuse(name + ".scales", s, want, u8)
        if not s.is_contiguous():
            raise PiError(PI_ERR_ARG, f"{name}.scales are not packed")
        return codes, s.data_ptr(), ld

    @staticmethod
    def _mx_dims(name, q):
        if not isinstance(q, MxMatrix):
            raise PiError(PI_ERR_ARG, f"{name} is not an MxMatrix")
        return q.shape

    def mx_empty(self, rows: int, cols: int, kind: int) -> MxMatrix:
        """A matrix for a call to write."""
        if kind != PI_MX8 and kind != PI_MX4:
            raise PiError(PI_ERR_ARG, f"kind {kind} is not PI_MX8 or PI_MX4")
        torch = _torch or _import_torch()
        B, dev = (cols + 127) // 128, self.torch_device
        return MxMatrix(torch.empty((rows, B * (128 if kind == PI_MX8 else 64)), dtype=torch.uint8, device=dev),
                        torch.empty(((rows + 127) // 128, B, 32, 4, 4), dtype=torch.uint8, device=dev), cols, kind)

    def _mx_out(self, name, q, rows, cols, kind):
        """(q or a new matrix, and what _mx says of it)"""
        if q is not None:
            return q, *self._mx(name, q, rows, cols, kind)
        q = self.mx_empty(rows, cols, kind)
        return q, q.codes.data_ptr(), q.scales.data_ptr(), 0

    def _out(self, name, t, shape, dtype):
        """(t or a new tensor, and what _at says of it)"""
        if t is not None:
            return t, *self._at(name, t, shape, dtype)
        t = (_torch or _import_torch()).empty(shape, dtype=dtype, device=self.torch_device)
        return t, t.data_ptr(), 0

    def mx_quantize(self, x, kind: int = PI_MX8, out: MxMatrix | None = None) -> MxMatrix:
        """x (float16, bfloat16 or float32 rows) in blocks of 32 columns that
        share a scale; elements of 8 (PI_MX8) or 4 bits (PI_MX4)."""
        code = self._code(x.dtype)
        T, K = self._dims("x", x)
        px, ldx = self._at("x", x, (T, K), x.dtype)
        out, pc, ps, ldq = self._mx_out("out", out, T, K, kind)
        desc, _ = self._plan(pi_mx_desc, (T, K, kind, code, ldx, ldq), None)
        q = pi_mx(pc, ps)
        self._s()
        rc = _lib.pi_mx_quantize(self.handle, ctypes.addressof(desc), px, ctypes.addressof(q))
        if rc:
            _check(self.handle, rc, "pi_mx_quantize")
        return out

    def mx_dequantize(self, q: MxMatrix, dtype=None, out=None):
        """The values of q in `dtype` (bfloat16 unless given, or out's)."""
        T, K = self._mx_dims("q", q)
        if dtype is None:
            dtype = (_torch or _import_torch()).bfloat16 if out is None else out.dtype
        code = self._code(dtype)
        pc, ps, ldq = self._mx("q", q, T, K)
        out, py, ldy = self._out("out", out, (T, K), dtype)
        desc, _ = self._plan(pi_mx_desc, (T, K, q.kind, code, ldy, ldq), None)
        m = pi_mx(pc, ps)
        self._s()
        rc = _lib.pi_mx_dequantize(self.handle, ctypes.addressof(desc), ctypes.addressof(m), py)
        if rc:
            _check(self.handle, rc, "pi_mx_dequantize")
        return out

    def mx_linear(self, x: MxMatrix, w: MxMatrix, b=None, *, fn=PI_FN_NONE, scale=1.0, residual=None, dtype=None, y=None):
        """y = residual + scale * fn(x W^T + b) of microscaled x and W (kinds
        8 and 4, 8 and 8, or 4 and 4 bits).  dtype: of b, and of y unless
        a residual or y says otherwise (float32 residual stream); bfloat16
        unless given."""
        T, K = self._mx_dims("x", x)
        N = self._mx_dims("w", w)[0]
        if dtype is None:
            t = b if b is not None else residual if residual is not None else y
            torch = _torch or _import_torch()
            dtype = torch.bfloat16 if t is None or t.dtype == torch.float32 else t.dtype
        code = self._code16(dtype)
        ydt = y.dtype if y is not None else dtype if residual is None else residual.dtype
        out = self._code(ydt)
        pxc, pxs, ldx = self._mx("x", x, T, K)
        pwc, pws, ldw = self._mx("w", w, N, K)
        pb = 0 if b is None else self._at("b", b, (N,), dtype)[0]
        pr, ldr = (0, 0) if residual is None else self._at("residual", residual, (T, N), ydt)
        y, py, ldy = self._out("y", y, (T, N), ydt)
        desc, n = self._plan(pi_mx_linear_desc, (T, K, N, x.kind, w.kind, code, out, fn, scale, ldx, ldw, ldr, ldy),
                             pi_mx_linear_workspace)
        mx, mw = pi_mx(pxc, pxs), pi_mx(pwc, pws)
        ws, pw = self._ws(n)
        self._s()
        rc = _lib.pi_mx_linear(self.handle, ctypes.addressof(desc), ctypes.addressof(mx), ctypes.addressof(mw), pb, pr, py, pw, n)
        if rc:
            _check(self.handle, rc, "pi_mx_linear")
        return y

    def mx_gated_ffn(self, x: MxMatrix, w_gate, w_up: MxMatrix, w_down: MxMatrix, b_gate=None, b_up=None, b_down=None, *,
                     fn=PI_FN_RELU, dtype=None, y=None):
        """y = Q(fn(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd of microscaled x
        and weights; Q quantises to x's kind.  w_gate None: fn(x Wu^T + bu)."""
        T, d = self._mx_dims("x", x)
        n = self._mx_dims("w_up", w_up)[0]
        if dtype is None:
            t = next((v for v in (b_gate, b_up, b_down, y) if v is not None), None)
            dtype = (_torch or _import_torch()).bfloat16 if t is None else t.dtype
        code = self._code16(dtype)
        pxc, pxs, ldx = self._mx("x", x, T, d)
        gc, gs, ldg = self._mx("w_gate", w_gate, n, d, w_up.kind)
        uc, us, ldu = self._mx("w_up", w_up, n, d)
        dc, ds, ldd = self._mx("w_down", w_down, d, n, w_up.kind)
        y, py, ldy = self._out("y", y, (T, d), dtype)
        pbg, pbu = self._at("b_gate", b_gate, (n,), dtype)[0], self._at("b_up", b_up, (n,), dtype)[0]
        pbd = self._at("b_down", b_down, (d,), dtype)[0]
        desc, nb = self._plan(pi_mx_gated_ffn_desc, (T, d, n, x.kind, w_up.kind, code, fn, w_gate is not None, ldx, ldg, ldu,
                                                     ldd, ldy), pi_mx_gated_ffn_workspace)
        wts, mx = pi_mx_gated_ffn_weights(gc, gs, uc, us, dc, ds, pbg, pbu, pbd), pi_mx(pxc, pxs)
        ws, pws = self._ws(nb)
        self._s()
        rc = _lib.pi_mx_gated_ffn(self.handle, ctypes.addressof(desc), ctypes.addressof(wts), ctypes.addressof(mx), py, pws, nb)
        if rc:
            _check(self.handle, rc, "pi_mx_gated_ffn")
        return y

    def norm_residual_mx(self, x, y=None, gate=None, *, kind: int = PI_MX8, pre=PI_NORM_RMS, post=PI_NORM_NONE, w_pre=None,
                         b_pre=None, w_post=None, b_post=None, res_scale=1.0, branch_scale=1.0, gate_rows=0, eps=1e-5,
                         dtype=None, x_out=None, h: MxMatrix | None = None):
        """``norm_residual`` with h quantised to `kind`: (x', h)."""
        xdt = x.dtype
        xcode = self._code(xdt)
        if y is not None:
            dtype = y.dtype
        elif dtype is None:
            dtype = next((v.dtype for v in (w_pre, b_pre) if v is not None),
                         (_torch or _import_torch()).bfloat16 if xcode == PI_F32 else xdt)
        code = self._code16(dtype)
        T, d = self._dims("x", x)
        px, ldx = self._at("x", x, (T, d), dtype if xcode != PI_F32 else xdt)
        py, ldy = self._at("y", y, (T, d), dtype)
        pg, ldg = self._at("gate", gate, (1 if gate_rows == 0 else -(-T // max(gate_rows, 1)), d), dtype)
        x_out, po, ldo = self._out("x_out", x_out, (T, d), xdt)
        h, hc, hs, ldh = self._mx_out("h", h, T, d, kind)
        par = pi_norm_residual_params(self._at("w_pre", w_pre, (d,), dtype)[0], self._at("b_pre", b_pre, (d,), dtype)[0],
                                      self._at("w_post", w_post, (d,), dtype)[0], self._at("b_post", b_post, (d,), dtype)[0])
        desc, _ = self._plan(pi_norm_residual_desc, (T, d, xcode, code, code, pre, post, gate_rows, res_scale, branch_scale,
                                                     eps, ldx, ldo, ldy, ldh, ldg), None)
        mh = pi_mx(hc, hs)
        self._s()
        rc = _lib.pi_norm_residual_mx(self.handle, ctypes.addressof(desc), kind, ctypes.addressof(par), px, py, pg, po,
                                      ctypes.addressof(mh))
        if rc:
            _check(self.handle, rc, "pi_norm_residual_mx")
        return x_out, h

    def set_trace(self, x_trace=None, xhat_trace=None, idx_trace=None, count_trace=None) -> None:
        pi_set_trace(self.handle, x_trace, xhat_trace, idx_trace, count_trace)

    def sync_status(self) -> int:
        self._s()
        return pi_sync_status(self.handle)

    def check(self) -> None:
        rc = self.sync_status()
        if rc:
            raise PiError(rc, pi_last_error(self.handle))
