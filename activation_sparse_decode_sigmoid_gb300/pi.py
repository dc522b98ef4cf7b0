"""Thin Python binding of libpi (include/pi.h): same entry-point names,
argument marshalling only.  Every step of the hot path runs in the library's
CUDA kernels; there is no CPU fallback.  If ``_build/libpi.so`` is missing this
module raises on first use -- build it with
``python -m activation_sparse_decode_sigmoid_gb300.build``.

Tensors are torch tensors on the context's device (PyTorch supplies device
memory and streams only).  16-bit data may be passed as float16 / bfloat16 or
as int16 / uint16 views of the bit patterns.  Every compute call is issued on
torch's current CUDA stream.
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
PI_F16, PI_BF16, PI_Q4_0, PI_F32 = 0, 1, 2, 3
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
           "pi_norm_residual_bwd")


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
                                ("ldx", "ldxo", "ldy", "ldh", "ldgate"))
pi_norm_residual_params = _struct("pi_norm_residual_params", ptr=("w_pre", "b_pre", "w_post", "b_post"))
pi_norm_residual_grads = _struct("pi_norm_residual_grads",
                                 ptr=("dx", "dy", "dgate", "dw_pre", "db_pre", "dw_post", "db_post"))


_lib = None


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


def _stream_ptr(device) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


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


# ---------------------------------------------------------------- convenience wrapper
class Context:
    """Owns a pi_ctx; every call runs on torch's current stream of `device`."""

    def __init__(self, device: int = 0, max_layers: int = 1, max_batch: int = 1):
        import torch
        self.device = device
        self.torch_device = torch.device("cuda", device)
        self.max_layers, self.max_batch = max_layers, max_batch
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
        pi_set_stream(self.handle, _stream_ptr(self.torch_device))

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
    def _args(self, dtype, **tensors):
        """Checks the tensors of a call: on the context's device, of `dtype`
        (or, for names ending in an underscore, also float32), rows of
        consecutive elements.  True if a base is not 16-byte aligned."""
        import torch
        if dtype not in (torch.float16, torch.bfloat16):
            raise PiError(PI_ERR_ARG, f"dtype {dtype} is not float16 or bfloat16")
        odd = False
        for name, t in tensors.items():
            if t is None:
                continue
            if t.device != self.torch_device:
                raise PiError(PI_ERR_ARG, f"{name.rstrip('_')} is on {t.device}, the context on {self.torch_device}")
            if t.dtype != dtype and not (name[-1] == "_" and t.dtype == torch.float32):
                raise PiError(PI_ERR_ARG, f"{name.rstrip('_')} is {t.dtype}, expected {dtype}")
            if t.dim() not in (1, 2):
                raise PiError(PI_ERR_SHAPE, f"{name.rstrip('_')} has {t.dim()} dimensions")
            if t.shape[-1] > 1 and t.stride(-1) != 1:
                raise PiError(PI_ERR_ARG, f"{name.rstrip('_')}: a row's elements are not consecutive")
            if t.dim() == 2 and t.shape[0] > 1 and t.stride(0) < t.shape[1]:
                raise PiError(PI_ERR_SHAPE, f"{name.rstrip('_')}: rows overlap (stride {t.stride(0)})")
            odd |= t.data_ptr() % 16 != 0
        return odd

    @staticmethod
    def _shape(name, t, *shape):
        if t is not None and tuple(t.shape) != shape:
            raise PiError(PI_ERR_SHAPE, f"{name} is {list(t.shape)}, expected {list(shape)}")

    @staticmethod
    def _packed(name, t):
        if t is not None and not t.is_contiguous():
            raise PiError(PI_ERR_ARG, f"{name} is not packed")

    @staticmethod
    def _ld(t) -> int:
        """Row stride of a matrix (a single row's own stride says nothing)."""
        return 0 if t is None or t.shape[0] <= 1 else t.stride(0)

    @staticmethod
    def _code(dtype) -> int:
        import torch
        return {torch.float16: PI_F16, torch.bfloat16: PI_BF16, torch.float32: PI_F32}[dtype]

    def _ws(self, n: int):
        import torch
        return torch.empty(n, dtype=torch.uint8, device=self.torch_device) if n else None

    def linear(self, x, w, b=None, *, fn=PI_FN_NONE, scale=1.0, residual=None, z=None, y=None):
        """y = residual + scale * fn(x W^T + b).  y is x's type, or the
        residual's (float32 residual stream); z, if given, receives
        x W^T + b for the backward pass."""
        import torch
        (T, K), N = x.shape, w.shape[0]
        if y is None:
            y = torch.empty((T, N), dtype=x.dtype if residual is None else residual.dtype, device=self.torch_device)
        odd = self._args(x.dtype, x=x, w=w, b=b, z=z, residual_=residual, y_=y)
        self._shape("w", w, N, K), self._shape("b", b, N), self._shape("z", z, T, N)
        self._shape("residual", residual, T, N), self._shape("y", y, T, N)
        if residual is not None and residual.dtype != y.dtype:
            raise PiError(PI_ERR_ARG, f"residual is {residual.dtype}, y {y.dtype}")
        code = self._code(x.dtype)
        desc = pi_linear_desc(T, K, N, code, self._code(y.dtype), code, fn, scale, odd, self._ld(x), self._ld(w),
                              self._ld(z), self._ld(residual), self._ld(y), 0, 0)
        self._s()
        n = pi_linear_workspace(self.handle, desc, False)
        pi_linear(self.handle, desc, x, w, b, residual, z, y, self._ws(n), n)
        return y

    def linear_bwd(self, dy, x, w, z=None, *, fn=PI_FN_NONE, scale=1.0, need=(True, True, True), dx=None, dw=None,
                   db=None, accumulate=False):
        """(dx, dw, db) of ``linear`` for the gradient dy of y (the residual's
        is dy itself).  need: which of them; buffers may be given, dw and db
        in x's type or float32, and are added to with `accumulate`."""
        import torch
        (T, K), N = x.shape, w.shape[0]
        new = lambda shape: torch.empty(shape, dtype=x.dtype, device=self.torch_device)
        if accumulate and any(n and g is None for n, g in zip(need[1:], (dw, db))):
            raise PiError(PI_ERR_ARG, "accumulate needs the buffers that it adds to")
        dx = (new((T, K)) if dx is None else dx) if need[0] else None
        dw = (new((N, K)) if dw is None else dw) if need[1] else None
        db = (torch.empty(N, dtype=x.dtype if dw is None else dw.dtype, device=self.torch_device) if db is None
              else db) if need[2] else None
        odd = self._args(x.dtype, dy_=dy, x=x, w=w, z=z, dx=dx, dw_=dw, db_=db)
        self._shape("dy", dy, T, N), self._shape("w", w, N, K), self._shape("z", z, T, N), self._shape("dx", dx, T, K)
        self._shape("dw", dw, N, K), self._shape("db", db, N)
        if dw is not None and db is not None and dw.dtype != db.dtype:
            raise PiError(PI_ERR_ARG, f"dw is {dw.dtype}, db {db.dtype}")
        grad = dw if dw is not None else db
        code = self._code(x.dtype)
        desc = pi_linear_desc(T, K, N, code, self._code(dy.dtype), code if grad is None else self._code(grad.dtype), fn,
                              scale, odd, self._ld(x), self._ld(w), self._ld(z), 0, self._ld(dy), self._ld(dx),
                              self._ld(dw))
        self._s()
        n = pi_linear_workspace(self.handle, desc, True)
        pi_linear_bwd(self.handle, desc, dy, x, w, z, dx, dw, db, accumulate, self._ws(n), n)
        return dx, dw, db

    def gated_ffn_save(self, x, w_gate, w_up):
        """Buffers (g, u, a) for ``gated_ffn`` to leave for its backward pass,
        [T][n] with rows that start on 128-byte boundaries (g None if not gated)."""
        import torch
        T, n = x.shape[0], w_up.shape[0]
        new = lambda: torch.empty((T, (n + 63) // 64 * 64), dtype=x.dtype, device=self.torch_device)[:, :n]
        return (new() if w_gate is not None else None), new(), new()

    def _ffn_desc(self, x, w_gate, w_up, w_down, g, u, a, y, fn, grad_code, odd):
        T, d = x.shape
        n = w_up.shape[0]
        for name, t, shape in (("w_gate", w_gate, (n, d)), ("w_up", w_up, (n, d)), ("w_down", w_down, (d, n)),
                               ("g", g, (T, n)), ("u", u, (T, n)), ("a", a, (T, n)), ("y", y, (T, d))):
            self._shape(name, t, *shape)
        return pi_gated_ffn_desc(T, d, n, self._code(x.dtype), grad_code, fn, w_gate is not None, odd, self._ld(x),
                                 self._ld(y), self._ld(w_gate), self._ld(w_up), self._ld(w_down), self._ld(g),
                                 self._ld(u), self._ld(a))

    def gated_ffn(self, x, w_gate, w_up, w_down, b_gate=None, b_up=None, b_down=None, *, fn=PI_FN_RELU, save=None,
                  y=None):
        """y = (fn(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd, weights in the
        model's layout; w_gate None: y = fn(x Wu^T + bu) Wd^T + bd.  save
        (``gated_ffn_save``) keeps g, u and a for the backward pass."""
        import torch
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=self.torch_device)
        g, u, a = save if save is not None else (None, None, None)
        odd = self._args(x.dtype, x=x, w_gate=w_gate, w_up=w_up, w_down=w_down, b_gate=b_gate, b_up=b_up, b_down=b_down,
                         g=g, u=u, a=a, y=y)
        desc = self._ffn_desc(x, w_gate, w_up, w_down, g, u, a, y, fn, self._code(x.dtype), odd)
        self._shape("b_gate", b_gate, desc.n), self._shape("b_up", b_up, desc.n), self._shape("b_down", b_down, desc.d)
        self._s()
        n = pi_gated_ffn_workspace(self.handle, desc, False)
        ws = pi_gated_ffn_weights(*map(_ptr, (w_gate, w_up, w_down, b_gate, b_up, b_down)))
        pi_gated_ffn(self.handle, desc, ws, x, pi_gated_ffn_save(*map(_ptr, (g, u, a))), y, self._ws(n), n)
        return y

    def gated_ffn_bwd(self, dy, x, w_gate, w_up, w_down, save, *, fn=PI_FN_RELU, need_dx=True, weight_grads=True,
                      bias_grads=True, grads=None, accumulate=False):
        """Gradients of ``gated_ffn`` for the gradient dy of y, as a dict with
        keys dx, w_gate, w_up, w_down, b_gate, b_up, b_down (None: not
        wanted).  grads: the parameter gradients' buffers by the same keys,
        packed, in x's type or float32 (all alike), used instead of new ones
        and added to with `accumulate`; then only the given ones are computed."""
        import torch
        g, u, a = save
        T, d = x.shape
        n, gated = w_up.shape[0], w_gate is not None
        shapes = {"w_gate": (n, d), "w_up": (n, d), "w_down": (d, n), "b_gate": (n,), "b_up": (n,), "b_down": (d,)}
        if grads is None:
            if accumulate:
                raise PiError(PI_ERR_ARG, "accumulate needs the buffers that it adds to")
            want = {k: weight_grads if k[0] == "w" else bias_grads for k in shapes}
            grads = {k: torch.empty(s, dtype=x.dtype, device=self.torch_device) for k, s in shapes.items()
                     if want[k] and (gated or k[2:] != "gate")}
        out = {k: grads.get(k) for k in shapes}
        dx = torch.empty((T, d), dtype=x.dtype, device=self.torch_device) if need_dx else None
        odd = self._args(x.dtype, dy=dy, x=x, w_gate=w_gate, w_up=w_up, w_down=w_down, g=g, u=u, a=a,
                         **{k + "_": v for k, v in out.items()})
        for k, v in out.items():
            self._shape(k, v, *shapes[k]), self._packed(k, v)
        types = {v.dtype for v in out.values() if v is not None}
        if len(types) > 1:
            raise PiError(PI_ERR_ARG, f"gradient buffers of several types: {types}")
        if x.stride(0) != d and T > 1 and dx is not None:  # (x and dx share their stride)
            dx = torch.empty((T, x.stride(0)), dtype=x.dtype, device=self.torch_device)[:, :d]
        desc = self._ffn_desc(x, w_gate, w_up, w_down, g, u, a, dy, fn, self._code(types.pop() if types else x.dtype), odd)
        self._s()
        nb = pi_gated_ffn_workspace(self.handle, desc, True)
        ws = pi_gated_ffn_weights(*map(_ptr, (w_gate, w_up, w_down)), None, None, None)
        pi_gated_ffn_bwd(self.handle, desc, ws, x, dy, pi_gated_ffn_save(*map(_ptr, (g, u, a))), dx,
                         pi_gated_ffn_grads(*(_ptr(out[k]) for k in shapes)), accumulate, self._ws(nb), nb)
        return {"dx": dx, **out}

    def _norm_desc(self, x, dtype, gate, pre, post, gate_rows, res_scale, branch_scale, eps, grad_code, lds):
        T, d = x.shape
        rows = 1 if gate_rows == 0 else -(-T // max(gate_rows, 1))
        self._shape("gate", gate, rows, d)
        return pi_norm_residual_desc(T, d, self._code(x.dtype), self._code(dtype), grad_code, pre, post, gate_rows,
                                     res_scale, branch_scale, eps, *lds)

    def norm_residual(self, x, y=None, gate=None, *, pre=PI_NORM_RMS, post=PI_NORM_NONE, w_pre=None, b_pre=None,
                      w_post=None, b_post=None, res_scale=1.0, branch_scale=1.0, gate_rows=0, eps=1e-5, dtype=None,
                      x_out=None, h=None):
        """(x', h): x' = res_scale * x + branch_scale * gate * norm_post(y),
        h = norm_pre(x') in y's type (`dtype` without a y).  gate [rows][d]:
        token t uses row t // gate_rows, 0 = one row for all.  x_out may be x."""
        import torch
        dtype = y.dtype if y is not None else dtype or (x.dtype if x.dtype != torch.float32 else torch.bfloat16)
        T, d = x.shape
        if x_out is None:
            x_out = torch.empty((T, d), dtype=x.dtype, device=self.torch_device)
        if h is None and pre != PI_NORM_NONE:
            h = torch.empty((T, d), dtype=dtype, device=self.torch_device)
        self._args(dtype, x_=x, y=y, gate=gate, w_pre=w_pre, b_pre=b_pre, w_post=w_post, b_post=b_post, x_out_=x_out, h=h)
        if x_out.dtype != x.dtype:
            raise PiError(PI_ERR_ARG, f"x_out is {x_out.dtype}, x {x.dtype}")
        for name, t in (("y", y), ("x_out", x_out), ("h", h)):
            self._shape(name, t, T, d)
        for name, t in (("w_pre", w_pre), ("b_pre", b_pre), ("w_post", w_post), ("b_post", b_post)):
            self._shape(name, t, d)
        desc = self._norm_desc(x, dtype, gate, pre, post, gate_rows, res_scale, branch_scale, eps, self._code(dtype),
                               (self._ld(x), self._ld(x_out), self._ld(y), self._ld(h), self._ld(gate)))
        self._s()
        pi_norm_residual(self.handle, desc, pi_norm_residual_params(*map(_ptr, (w_pre, b_pre, w_post, b_post))), x, y,
                         gate, x_out, h)
        return x_out, h

    def norm_residual_bwd(self, dx_out, dh, x_out, y=None, gate=None, *, pre=PI_NORM_RMS, post=PI_NORM_NONE, w_pre=None,
                          b_pre=None, w_post=None, b_post=None, res_scale=1.0, branch_scale=1.0, gate_rows=0, eps=1e-5,
                          grads=None, accumulate=False):
        """Gradients of ``norm_residual`` for the gradients dx_out of x' (None:
        0) and dh of h, as a dict with keys dx, dy, gate, w_pre, b_pre,
        w_post, b_post; a parameter that was not given has none.  grads:
        buffers for gate and the parameters, packed, in h's type or float32
        (all alike), used instead of new ones and added to with `accumulate`."""
        import torch
        dtype = next((t.dtype for t in (dh, y) if t is not None), None)
        if dtype is None:
            raise PiError(PI_ERR_ARG, "neither dh nor y given")
        T, d = x_out.shape
        given = {"gate": gate, "w_pre": w_pre, "b_pre": b_pre, "w_post": w_post, "b_post": b_post}
        if grads is None:
            if accumulate:
                raise PiError(PI_ERR_ARG, "accumulate needs the buffers that it adds to")
            grads = {k: torch.empty(v.shape, dtype=dtype, device=self.torch_device) for k, v in given.items()
                     if v is not None}
        out = {k: grads.get(k) for k in given}
        dx = torch.empty((T, d), dtype=x_out.dtype, device=self.torch_device)
        # (y and dy share their stride)
        dy = None if y is None else torch.empty((T, max(d, self._ld(y))), dtype=dtype, device=self.torch_device)[:, :d]
        self._args(dtype, dx_out_=dx_out, dh=dh, x_out_=x_out, y=y, **given, **{"d" + k + "_": v for k, v in out.items()})
        for name, t in (("dx_out", dx_out), ("dh", dh), ("y", y)):
            self._shape(name, t, T, d)
        for k, v in out.items():
            self._shape("gradient of " + k, v, *(given[k].shape if given[k] is not None else (d,)))
            self._packed("gradient of " + k, v)
            if k != "gate":
                self._shape(k, given[k], d)
        if dx_out is not None and dx_out.dtype != x_out.dtype:
            raise PiError(PI_ERR_ARG, f"dx_out is {dx_out.dtype}, x_out {x_out.dtype}")
        if dx_out is not None and self._ld(dx_out) != self._ld(x_out):
            raise PiError(PI_ERR_ARG, "dx_out and x_out differ in their row stride")
        types = {v.dtype for v in out.values() if v is not None}
        if len(types) > 1:
            raise PiError(PI_ERR_ARG, f"gradient buffers of several types: {types}")
        desc = self._norm_desc(x_out, dtype, gate, pre, post, gate_rows, res_scale, branch_scale, eps,
                               self._code(types.pop() if types else dtype),
                               (0, self._ld(x_out), self._ld(y), self._ld(dh), self._ld(gate)))
        self._s()
        n = pi_norm_residual_bwd_workspace(self.handle, desc)
        pi_norm_residual_bwd(self.handle, desc, pi_norm_residual_params(*map(_ptr, (w_pre, b_pre, w_post, b_post))),
                             dx_out, dh, x_out, y, gate, pi_norm_residual_grads(_ptr(dx), _ptr(dy),
                                                                               *(_ptr(out[k]) for k in given)),
                             accumulate, self._ws(n), n)
        return {"dx": dx, "dy": dy, **out}

    def set_trace(self, x_trace=None, xhat_trace=None, idx_trace=None, count_trace=None) -> None:
        pi_set_trace(self.handle, x_trace, xhat_trace, idx_trace, count_trace)

    def sync_status(self) -> int:
        self._s()
        return pi_sync_status(self.handle)

    def check(self) -> None:
        rc = self.sync_status()
        if rc:
            raise PiError(rc, pi_last_error(self.handle))
