"""Python binding of libmok.so (the C ABI in include/mok.h).

Argument marshalling only: every step of the layer runs in the CUDA library.
Tensors are torch CUDA tensors; PyTorch supplies device memory and streams.
If the library or a CUDA device is missing, calls raise - there is no CPU
fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmok.so")

BF16, MXFP8 = 0, 1
OK, ERR_INVALID, ERR_CUDA, ERR_TIMEOUT, ERR_CAPACITY, ERR_UNSUPPORTED = range(6)
STATUS_NAMES = {0: "MOK_OK", 1: "MOK_ERR_INVALID", 2: "MOK_ERR_CUDA", 3: "MOK_ERR_TIMEOUT",
                4: "MOK_ERR_CAPACITY", 5: "MOK_ERR_UNSUPPORTED"}

# every function declared in include/mok.h
EXPORTS = ["mok_route_workspace_size", "mok_route_layout", "mok_packed_weights_size", "mok_pack_weights",
           "mok_workspace_size", "mok_saved_size", "mok_moe_forward", "mok_padded_rows_max", "mok_dispatch",
           "mok_expert_ffn", "mok_combine", "mok_moe_backward", "mok_device_status", "mok_status_string",
           "mok_version", "mok_route_layout_static", "mok_workspace_size_batches", "mok_moe_forward_batches",
           "mok_quantize_rows", "mok_dispatch_quantized", "mok_route_test_hook", "mok_ep_workspace_size",
           "mok_ep_dispatch", "mok_ep_push", "mok_packed_weights_bwd_size", "mok_pack_weights_bwd",
           "mok_dispatch_tokens", "mok_rmsnorm", "mok_rmsnorm_bwd_workspace_size", "mok_rmsnorm_backward",
           "mok_dequantize_rows", "mok_checkpoint_size", "mok_checkpoint_save", "mok_checkpoint_load",
           "mok_few_workspace_size", "mok_moe_few", "mok_sort_workspace_size", "mok_sort_layout", "mok_sort_rows",
           "mok_unsort_rows", "mok_unsort_rows_backward", "mok_head_workspace_size", "mok_head_loss",
           "mok_head_loss_backward", "mok_head_loss_train", "mok_grad_workspace_size", "mok_grad_norm",
           "mok_grad_clip"]

FLAG_MEGAKERNEL = 1
FLAG_GEMM_PAIRS = 2
FLAG_TRACE = 4
FLAG_MB_TOKEN_RANGES = 8
FLAG_ROW_TILES = 16
FLAG_TOKEN_TILES_BALANCED = 32
FLAG_NO_L2_PREFETCH = 64
FLAG_SWAPPED_TILES = 128
FLAG_TEST_WITHHOLD_PUBLISH = 256


class MokError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}")
        self.code = code


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("dtype", ctypes.c_int32), ("I_shared", ctypes.c_int32)]


class Config(ctypes.Structure):
    _fields_ = [("num_sms", ctypes.c_int32), ("timeout_ms", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("mover_ctas", ctypes.c_int32), ("minibatch_tokens", ctypes.c_int32), ("ring_rows", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 2)]


class Routing(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("row_src", ctypes.c_void_p), ("slot_row", ctypes.c_void_p)]


class FwdArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("packed", ctypes.c_void_p), ("packed_shared", ctypes.c_void_p),
                ("routing", Routing), ("out", ctypes.c_void_p), ("saved", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


class BwdArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("W_r", ctypes.c_void_p), ("W_gate", ctypes.c_void_p),
                ("W_up", ctypes.c_void_p), ("W_down", ctypes.c_void_p), ("packed", ctypes.c_void_p),
                ("dY", ctypes.c_void_p), ("routing", Routing), ("saved", ctypes.c_void_p),
                ("dX", ctypes.c_void_p), ("dW_gate", ctypes.c_void_p), ("dW_up", ctypes.c_void_p),
                ("dW_down", ctypes.c_void_p), ("dW_r", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t), ("packed_bwd", ctypes.c_void_p)]


class EpPeer(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("row_src", ctypes.c_void_p),
                ("partials", ctypes.c_void_p), ("T", ctypes.c_int32)]


class RmsNormArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("residual", ctypes.c_void_p),
                ("ldr", ctypes.c_int64), ("gain", ctypes.c_void_p), ("eps", ctypes.c_float), ("sum", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("y_q", ctypes.c_void_p), ("y_sf", ctypes.c_void_p),
                ("sum_q", ctypes.c_void_p), ("sum_sf", ctypes.c_void_p), ("rstd", ctypes.c_void_p)]


class RmsNormBwdArgs(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("sum", ctypes.c_void_p), ("sum_q", ctypes.c_void_p),
                ("sum_sf", ctypes.c_void_p), ("dsum", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("gain", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("dgain", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t), ("labels", ctypes.c_void_p),
                ("labels_i64", ctypes.c_int32), ("V", ctypes.c_int32)]


class FewArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("W_r", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("packed", ctypes.c_void_p), ("packed_shared", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t)]


class HeadArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("W", ctypes.c_void_p), ("labels", ctypes.c_void_p),
                ("labels_i64", ctypes.c_int32), ("piece", ctypes.c_int32), ("loss", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("dloss", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("dW_f32", ctypes.c_int32), ("accumulate", ctypes.c_int32), ("dx", ctypes.c_void_p),
                ("dW", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


class GradTensor(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("elem", ctypes.c_int32)]


EP_MAX_RANKS = 8
STATUS_BYTES = 256     # the status block at the start of a workspace
FEW_MAX_TOKENS = 128   # MOK_FEW_MAX_TOKENS
FEW_MAX_PAIRS = 2048   # MOK_FEW_MAX_PAIRS
_lock = threading.Lock()
_lib = None


def lib():
    """Load libmok.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libmok.so not built ({LIB_PATH}); run __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            PP = ctypes.POINTER(Problem)
            PC = ctypes.POINTER(Config)
            PR = ctypes.POINTER(Routing)
            L.mok_route_workspace_size.argtypes = [I32] * 4
            L.mok_route_workspace_size.restype = SZ
            L.mok_route_layout.argtypes = [P, P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, SZ, P]
            L.mok_route_layout_static.argtypes = [P, P, P, I32, I32, I32, I32, P, P, P, P, P, P, P]
            L.mok_packed_weights_size.argtypes = [I32] * 4
            L.mok_packed_weights_size.restype = SZ
            L.mok_pack_weights.argtypes = [I32, I32, I32, I32, P, P, P, P, SZ, P]
            L.mok_packed_weights_bwd_size.argtypes = [I32] * 4
            L.mok_packed_weights_bwd_size.restype = SZ
            L.mok_pack_weights_bwd.argtypes = [I32, I32, I32, I32, P, P, P, P, SZ, P]
            L.mok_workspace_size.argtypes = [PP, PC]
            L.mok_workspace_size.restype = SZ
            L.mok_saved_size.argtypes = [PP]
            L.mok_saved_size.restype = SZ
            L.mok_moe_forward.argtypes = [PP, ctypes.POINTER(FwdArgs), PC, P]
            L.mok_moe_forward_batches.argtypes = [PP, I32, ctypes.POINTER(FwdArgs), PC, P]
            L.mok_workspace_size_batches.argtypes = [PP, I32, PC]
            L.mok_workspace_size_batches.restype = SZ
            L.mok_padded_rows_max.argtypes = [I32, I32, I32]
            L.mok_padded_rows_max.restype = ctypes.c_int64
            L.mok_dispatch.argtypes = [PP, P, PR, P, P, P]
            L.mok_quantize_rows.argtypes = [P, I32, I32, P, P, P]
            L.mok_dispatch_tokens.argtypes = [PP, P, PR, P, P, P]
            L.mok_dispatch_quantized.argtypes = [PP, P, P, PR, P, P, P]
            L.mok_expert_ffn.argtypes = [PP, P, P, P, PR, P, P, P, PC, P, P]
            L.mok_combine.argtypes = [PP, P, P, P, P, P]
            L.mok_moe_backward.argtypes = [PP, ctypes.POINTER(BwdArgs), PC, P]
            L.mok_device_status.argtypes = [P, P, ctypes.POINTER(I32), I32]
            L.mok_route_test_hook.argtypes = [I32, I32]
            L.mok_ep_workspace_size.argtypes = [I32, I32]
            L.mok_ep_workspace_size.restype = SZ
            L.mok_ep_dispatch.argtypes = [I32, I32, I32, I32, I32, ctypes.POINTER(EpPeer), P, P, ctypes.c_int64, P, P,
                                          P, P, P, P, SZ, P]
            L.mok_ep_push.argtypes = [I32, I32, I32, I32, ctypes.POINTER(EpPeer), P, ctypes.c_int64, P, P, P, P]
            L.mok_rmsnorm.argtypes = [I32, I32, ctypes.POINTER(RmsNormArgs), P]
            L.mok_rmsnorm_bwd_workspace_size.argtypes = [I32, I32]
            L.mok_rmsnorm_bwd_workspace_size.restype = SZ
            L.mok_rmsnorm_backward.argtypes = [I32, I32, ctypes.POINTER(RmsNormBwdArgs), P]
            L.mok_dequantize_rows.argtypes = [P, P, I32, I32, P, P]
            L.mok_checkpoint_size.argtypes = [PP]
            L.mok_checkpoint_size.restype = SZ
            L.mok_checkpoint_save.argtypes = [PP, P, PR, P, P, SZ, P]
            L.mok_checkpoint_load.argtypes = [PP, P, SZ, PR, P, P, P]
            L.mok_few_workspace_size.argtypes = [PP, PC]
            L.mok_few_workspace_size.restype = SZ
            L.mok_moe_few.argtypes = [PP, ctypes.POINTER(FewArgs), PC, P]
            L.mok_sort_workspace_size.argtypes = [I32] * 3
            L.mok_sort_workspace_size.restype = SZ
            L.mok_sort_layout.argtypes = [P, I32, I32, I32, P, P, P, P, P, SZ, P]
            L.mok_sort_rows.argtypes = [P, ctypes.c_int64, P, I32, I32, I32, I32, P, P]
            L.mok_unsort_rows.argtypes = [P, P, P, I32, I32, I32, I32, P, P]
            L.mok_unsort_rows_backward.argtypes = [P, P, P, P, I32, I32, I32, I32, P, P, P]
            L.mok_head_workspace_size.argtypes = [I32] * 5 + [PC]
            L.mok_head_workspace_size.restype = SZ
            for name in ("mok_head_loss", "mok_head_loss_backward", "mok_head_loss_train"):
                getattr(L, name).argtypes = [I32, I32, I32, ctypes.POINTER(HeadArgs), PC, P]
            L.mok_grad_workspace_size.restype = SZ
            L.mok_grad_norm.argtypes = [I32, ctypes.POINTER(GradTensor), P, P, SZ, P]
            L.mok_grad_clip.argtypes = [I32, ctypes.POINTER(GradTensor), ctypes.c_double, P, P, SZ, P]
            L.mok_status_string.argtypes = [I32]
            L.mok_status_string.restype = ctypes.c_char_p
            L.mok_version.restype = ctypes.c_char_p
            for name in ("mok_route_layout", "mok_route_layout_static", "mok_pack_weights", "mok_moe_forward",
                         "mok_moe_forward_batches", "mok_dispatch", "mok_quantize_rows", "mok_dispatch_quantized",
                         "mok_expert_ffn", "mok_combine", "mok_moe_backward", "mok_device_status", "mok_route_test_hook",
                         "mok_ep_dispatch", "mok_ep_push", "mok_pack_weights_bwd", "mok_dispatch_tokens", "mok_rmsnorm",
                         "mok_rmsnorm_backward", "mok_dequantize_rows", "mok_checkpoint_save", "mok_checkpoint_load",
                         "mok_moe_few", "mok_sort_layout", "mok_sort_rows", "mok_unsort_rows",
                         "mok_unsort_rows_backward", "mok_head_loss", "mok_head_loss_backward",
                         "mok_head_loss_train", "mok_grad_norm", "mok_grad_clip"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:   # the raw handle: building a Stream object costs 2.5 us a call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _allocating(stream):
    """Context for what a call on `stream` allocates, so that it is not handed to another stream's work once the call
    has dropped it, while its kernels still use it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _check(rc, what):
    if rc != OK:
        raise MokError(rc, what)


def _bf16(t):
    assert t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous(), "bf16 contiguous CUDA tensor expected"
    return t


def make_problem(T, H, I, E, k, dtype=BF16, I_shared=0) -> Problem:
    return Problem(T, H, I, E, k, dtype, I_shared)


def make_config(num_sms=0, timeout_ms=0, flags=0, mover_ctas=0, minibatch_tokens=0, ring_rows=0) -> Config:
    return Config(num_sms, timeout_ms, flags, mover_ctas, minibatch_tokens, ring_rows)


# --------------------------------------------------------------------------- sizes

def route_workspace_size(T, H, E, k) -> int:
    return int(lib().mok_route_workspace_size(T, H, E, k))


def packed_weights_size(E, H, I, dtype) -> int:
    return int(lib().mok_packed_weights_size(E, H, I, dtype))


def workspace_size(p: Problem, cfg: Config | None = None) -> int:
    return int(lib().mok_workspace_size(ctypes.byref(p), ctypes.byref(cfg) if cfg else None))


def workspace_size_batches(p: Problem, nbatch: int, cfg: Config | None = None) -> int:
    return int(lib().mok_workspace_size_batches(ctypes.byref(p), nbatch, ctypes.byref(cfg) if cfg else None))


def saved_size(p: Problem) -> int:
    return int(lib().mok_saved_size(ctypes.byref(p)))


def padded_rows_max(T, E, k) -> int:
    return int(lib().mok_padded_rows_max(T, E, k))


def version() -> str:
    return lib().mok_version().decode()


# --------------------------------------------------------------------------- calls

def alloc_bytes(n, device="cuda"):
    """Device buffer of n bytes, 1024-byte aligned (torch's caching allocator
    returns 512-byte aligned blocks; one extra KiB is sliced off the front)."""
    raw = torch.empty(max(int(n), 1) + 1024, dtype=torch.uint8, device=device)
    off = (-raw.data_ptr()) % 1024
    return raw[off:off + max(int(n), 1)]


def route_layout(x, W_r, k, bias=None, out=None, workspace=None, stream=None):
    """Router + top-k + layout. Returns a dict of device tensors (new ones are `stream`'s in the allocator)."""
    _bf16(x)
    T, H = x.shape
    E = W_r.shape[1]
    dev = x.device
    if out is None or workspace is None:
        with _allocating(stream):
            if out is None:
                out = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device=dev),
                           topk_w=torch.empty((T, k), dtype=torch.float32, device=dev),
                           counts=torch.empty(E, dtype=torch.int32, device=dev),
                           offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                           row_src=torch.empty(T * k, dtype=torch.int32, device=dev),
                           slot_row=torch.empty(T * k, dtype=torch.int32, device=dev))
            if workspace is None:
                workspace = alloc_bytes(route_workspace_size(T, H, E, k), dev)
    rc = lib().mok_route_layout(_ptr(x), _ptr(W_r), _ptr(bias), T, H, E, k, _ptr(out["topk_idx"]),
                                _ptr(out["topk_w"]), _ptr(out["counts"]), _ptr(out["offsets"]),
                                _ptr(out["row_src"]), _ptr(out["slot_row"]), _ptr(workspace),
                                workspace.numel(), _stream(stream))
    _check(rc, "mok_route_layout")
    return out


ROUTE_STATIC_SCRATCH_BYTES = 8 << 20  # MOK_ROUTE_STATIC_SCRATCH_BYTES


def route_layout_static(x, W_r, k, bias=None, out=None, stream=None):
    """Routing with the library's own scratch array: no workspace argument,
    nothing allocated by the library (the outputs are still the caller's)."""
    _bf16(x)
    T, H = x.shape
    E = W_r.shape[1]
    dev = x.device
    if out is None:
        out = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device=dev),
                   topk_w=torch.empty((T, k), dtype=torch.float32, device=dev),
                   counts=torch.empty(E, dtype=torch.int32, device=dev),
                   offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                   row_src=torch.empty(max(T * k, 1), dtype=torch.int32, device=dev),
                   slot_row=torch.empty(max(T * k, 1), dtype=torch.int32, device=dev))
    rc = lib().mok_route_layout_static(_ptr(x), _ptr(W_r), _ptr(bias), T, H, E, k, _ptr(out["topk_idx"]),
                                       _ptr(out["topk_w"]), _ptr(out["counts"]), _ptr(out["offsets"]),
                                       _ptr(out["row_src"]), _ptr(out["slot_row"]), _stream(stream))
    _check(rc, "mok_route_layout_static")
    return out


def routing_struct(r) -> Routing:
    return Routing(r["topk_idx"].data_ptr(), r["topk_w"].data_ptr(), r["counts"].data_ptr(),
                   r["offsets"].data_ptr(), r["row_src"].data_ptr(), r["slot_row"].data_ptr())


def pack_weights(Wg, Wu, Wd, dtype, packed=None, stream=None):
    E, H, I = Wg.shape
    n = packed_weights_size(E, H, I, dtype)
    if n == 0:
        raise MokError(ERR_INVALID, "mok_packed_weights_size")
    if packed is None:
        packed = alloc_bytes(n, Wg.device)
    rc = lib().mok_pack_weights(E, H, I, dtype, _ptr(_bf16(Wg)), _ptr(_bf16(Wu)), _ptr(_bf16(Wd)), _ptr(packed),
                                packed.numel(), _stream(stream))
    _check(rc, "mok_pack_weights")
    return packed


def pack_weights_bwd(Wg, Wu, Wd, dtype, packed_bwd=None, stream=None):
    """The MXFP8 backward's weight copies (None for BF16)."""
    E, H, I = Wg.shape
    n = int(lib().mok_packed_weights_bwd_size(E, H, I, dtype))
    if n == 0:
        return None
    if packed_bwd is None:
        packed_bwd = alloc_bytes(n, Wg.device)
    rc = lib().mok_pack_weights_bwd(E, H, I, dtype, _ptr(_bf16(Wg)), _ptr(_bf16(Wu)), _ptr(_bf16(Wd)),
                                    _ptr(packed_bwd), packed_bwd.numel(), _stream(stream))
    _check(rc, "mok_pack_weights_bwd")
    return packed_bwd


def moe_forward(p: Problem, x, packed, routing, out, workspace, saved=None, packed_shared=None,
                cfg: Config | None = None, stream=None):
    a = FwdArgs(x.data_ptr(), packed.data_ptr(), packed_shared.data_ptr() if packed_shared is not None else None,
                routing_struct(routing), out.data_ptr(), saved.data_ptr() if saved is not None else None,
                workspace.data_ptr(), workspace.numel())
    rc = lib().mok_moe_forward(ctypes.byref(p), ctypes.byref(a), ctypes.byref(cfg) if cfg else None, _stream(stream))
    _check(rc, "mok_moe_forward")
    return out


def moe_forward_batches(p: Problem, xs, packed, routings, outs, workspace, packed_shared=None,
                        cfg: Config | None = None, stream=None):
    """One megakernel launch over len(xs) macro-batches (same weights)."""
    n = len(xs)
    arr = (FwdArgs * n)()
    for b in range(n):
        arr[b] = FwdArgs(xs[b].data_ptr(), packed.data_ptr(),
                         packed_shared.data_ptr() if packed_shared is not None else None,
                         routing_struct(routings[b]), outs[b].data_ptr(), None, workspace.data_ptr(),
                         workspace.numel())
    rc = lib().mok_moe_forward_batches(ctypes.byref(p), n, arr, ctypes.byref(cfg) if cfg else None, _stream(stream))
    _check(rc, "mok_moe_forward_batches")
    return outs


def moe_backward(p: Problem, x, W_r, Wg, Wu, Wd, packed, dY, routing, saved, grads, workspace,
                 cfg: Config | None = None, stream=None, packed_bwd=None):
    """grads: dict with dX, dW_gate, dW_up, dW_down, dW_r (preallocated)."""
    a = BwdArgs(x.data_ptr(), W_r.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(), packed.data_ptr(),
                dY.data_ptr(), routing_struct(routing), saved.data_ptr(), grads["dX"].data_ptr(),
                grads["dW_gate"].data_ptr(), grads["dW_up"].data_ptr(), grads["dW_down"].data_ptr(),
                grads["dW_r"].data_ptr(), workspace.data_ptr(), workspace.numel(),
                packed_bwd.data_ptr() if packed_bwd is not None else None)
    rc = lib().mok_moe_backward(ctypes.byref(p), ctypes.byref(a), ctypes.byref(cfg) if cfg else None,
                                _stream(stream))
    _check(rc, "mok_moe_backward")
    return grads


def dispatch(p: Problem, x, routing, A, A_sf=None, stream=None):
    rs = routing_struct(routing)
    rc = lib().mok_dispatch(ctypes.byref(p), _ptr(x), ctypes.byref(rs), _ptr(A), _ptr(A_sf), _stream(stream))
    _check(rc, "mok_dispatch")


def dispatch_tokens(p: Problem, x, routing, A, A_sf, stream=None):
    rs = routing_struct(routing)
    rc = lib().mok_dispatch_tokens(ctypes.byref(p), _ptr(x), ctypes.byref(rs), _ptr(A), _ptr(A_sf), _stream(stream))
    _check(rc, "mok_dispatch_tokens")


def quantize_rows(x, x_q, x_sf, stream=None):
    T, H = x.shape
    rc = lib().mok_quantize_rows(_ptr(x), T, H, _ptr(x_q), _ptr(x_sf), _stream(stream))
    _check(rc, "mok_quantize_rows")


def dispatch_quantized(p: Problem, x_q, x_sf, routing, A, A_sf, stream=None):
    rs = routing_struct(routing)
    rc = lib().mok_dispatch_quantized(ctypes.byref(p), _ptr(x_q), _ptr(x_sf), ctypes.byref(rs), _ptr(A), _ptr(A_sf),
                                      _stream(stream))
    _check(rc, "mok_dispatch_quantized")


def expert_ffn(p: Problem, A, A_sf, packed, routing, h, h_sf, partials, workspace, cfg: Config | None = None,
               stream=None):
    rs = routing_struct(routing)
    rc = lib().mok_expert_ffn(ctypes.byref(p), _ptr(A), _ptr(A_sf), _ptr(packed), ctypes.byref(rs), _ptr(h),
                              _ptr(h_sf), _ptr(partials), ctypes.byref(cfg) if cfg else None, _ptr(workspace),
                              _stream(stream))
    _check(rc, "mok_expert_ffn")


def combine(p: Problem, partials, topk_w, out, shared=None, stream=None):
    rc = lib().mok_combine(ctypes.byref(p), _ptr(partials), _ptr(topk_w), _ptr(shared), _ptr(out), _stream(stream))
    _check(rc, "mok_combine")


# --------------------------------------------------------------------------- pre-norm

def _addr(t):
    return None if t is None else t.data_ptr()


# The checks of tensors raise by themselves: a kernel that is given another tensor reads out of range, also where
# Python drops assert statements (-O).

def _dense(name, t, dtype, *shape):
    """t (or None) is a contiguous CUDA tensor of this type and shape."""
    if t is not None and not (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()):
        raise AssertionError(f"{name}: contiguous {dtype} CUDA tensor {list(shape)} expected")


def _here(name, t, device, dtype, *shape):
    """The same, on this device (the current one)."""
    if t is not None and not (t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous()):
        raise AssertionError(f"{name}: contiguous {dtype} tensor {list(shape)} on CUDA device {device} expected")


def _scratch(t, device):
    """The address of a workspace on this device."""
    if t.get_device() != device:
        raise AssertionError(f"workspace: tensor on CUDA device {device} expected")
    return t.data_ptr()


def _rows(name, t, T, H):
    """Row pitch of bf16 rows whose elements are adjacent (of a single row: H, whatever view it is)."""
    pitch, step = t.stride()
    if not (t.dtype is torch.bfloat16 and step == 1 and t.shape == (T, H) and t.is_cuda):
        raise AssertionError(f"{name}: bf16 CUDA tensor [{T}, {H}] with adjacent row elements expected")
    return pitch if T > 1 else H


def rmsnorm(x, gain, residual=None, eps=1e-6, sum=None, y=None, y_q=None, y_sf=None, sum_q=None, sum_sf=None,
            rstd=None, stream=None):
    """Residual's addition and root-mean-square norm, into the outputs given
    (see mok_rmsnorm). x and residual may be row-strided views."""
    T, H = x.shape
    _dense("sum", sum, torch.bfloat16, T, H)
    _dense("y", y, torch.bfloat16, T, H)
    if y_q is not None or y_sf is not None:
        _dense("y_q", y_q, torch.uint8, T, H)
        _dense("y_sf", y_sf, torch.uint8, T, H // 32)
    if sum_q is not None or sum_sf is not None:
        _dense("sum_q", sum_q, torch.uint8, T, H)
        _dense("sum_sf", sum_sf, torch.uint8, T, H // 32)
    _dense("gain", gain, torch.float32, H)
    _dense("rstd", rstd, torch.float32, T)
    a = RmsNormArgs(x.data_ptr(), _rows("x", x, T, H), _addr(residual),
                    0 if residual is None else _rows("residual", residual, T, H), gain.data_ptr(), eps, _addr(sum),
                    _addr(y), _addr(y_q), _addr(y_sf), _addr(sum_q), _addr(sum_sf), _addr(rstd))
    _check(lib().mok_rmsnorm(T, H, ctypes.byref(a), _stream(stream)), "mok_rmsnorm")


def rmsnorm_bwd_workspace_size(T, H) -> int:
    return int(lib().mok_rmsnorm_bwd_workspace_size(T, H))


def rmsnorm_backward(dy, gain, rstd, dx, dgain, workspace, s=None, s_q=None, s_sf=None, dsum=None, stream=None,
                     labels=None, V=0):
    """Gradients of rmsnorm from the forward's sum, in BF16 (s) or as MXFP8 rows (s_q, s_sf). labels [T] (int32 or
    int64, with s): rows whose label is outside 0..V-1 count as zeros, whatever they hold."""
    T, H = dy.shape
    _dense("dy", dy, torch.bfloat16, T, H)
    _dense("dx", dx, torch.bfloat16, T, H)
    _dense("s", s, torch.bfloat16, T, H)
    _dense("dsum", dsum, torch.bfloat16, T, H)
    if s_q is not None or s_sf is not None:
        _dense("s_q", s_q, torch.uint8, T, H)
        _dense("s_sf", s_sf, torch.uint8, T, H // 32)
    _dense("gain", gain, torch.float32, H)
    _dense("dgain", dgain, torch.float32, H)
    _dense("rstd", rstd, torch.float32, T)
    i64 = False
    if labels is not None:
        i64 = labels.dtype is torch.int64
        _dense("labels", labels, torch.int64 if i64 else torch.int32, T)
    a = RmsNormBwdArgs(dy.data_ptr(), _addr(s), _addr(s_q), _addr(s_sf), _addr(dsum), rstd.data_ptr(),
                       gain.data_ptr(), dx.data_ptr(), dgain.data_ptr(), workspace.data_ptr(), workspace.numel(),
                       _addr(labels), i64, V)
    _check(lib().mok_rmsnorm_backward(T, H, ctypes.byref(a), _stream(stream)), "mok_rmsnorm_backward")


def dequantize_rows(x_q, x_sf, x, stream=None):
    """BF16 values of MXFP8 rows (the way back from quantize_rows)."""
    T, H = x.shape
    _dense("x", x, torch.bfloat16, T, H)
    _dense("x_q", x_q, torch.uint8, T, H)
    _dense("x_sf", x_sf, torch.uint8, T, H // 32)
    _check(lib().mok_dequantize_rows(_ptr(x_q), _ptr(x_sf), T, H, _ptr(x), _stream(stream)), "mok_dequantize_rows")


# --------------------------------------------------------------------------- the layer for a few tokens

def few_tokens_ok(T, k) -> bool:
    """Whether moe_few takes T tokens with k experts each."""
    return T <= FEW_MAX_TOKENS and T * k <= FEW_MAX_PAIRS


def few_workspace_size(p: Problem, cfg: Config | None = None) -> int:
    return int(lib().mok_few_workspace_size(ctypes.byref(p), ctypes.byref(cfg) if cfg else None))


def moe_few(p: Problem, x, W_r, packed, out, workspace, bias=None, packed_shared=None, topk_idx=None, topk_w=None,
            cfg: Config | None = None, stream=None):
    """The whole layer for p.T <= FEW_MAX_TOKENS tokens (p.T * p.k <= FEW_MAX_PAIRS)."""
    T, H, E, k = p.T, p.H, p.E, p.k
    _dense("x", x, torch.bfloat16, T, H)
    _dense("out", out, torch.bfloat16, T, H)
    _dense("W_r", W_r, torch.float32, H, E)
    _dense("topk_idx", topk_idx, torch.int32, T, k)
    _dense("topk_w", topk_w, torch.float32, T, k)
    _dense("bias", bias, torch.float32, E)
    a = FewArgs(x.data_ptr(), W_r.data_ptr(), _addr(bias), packed.data_ptr(), _addr(packed_shared), out.data_ptr(),
                _addr(topk_idx), _addr(topk_w), workspace.data_ptr(), workspace.numel())
    _check(lib().mok_moe_few(ctypes.byref(p), ctypes.byref(a), ctypes.byref(cfg) if cfg else None, _stream(stream)),
           "mok_moe_few")
    return out


# --------------------------------------------------------------------------- 8-bit training context

def checkpoint_size(p: Problem) -> int:
    return int(lib().mok_checkpoint_size(ctypes.byref(p)))


def checkpoint_save(p: Problem, x, routing, saved, ckpt, stream=None):
    """MXFP8 copy of a training forward's context (x, pre-activations, partials)."""
    _dense("x", x, torch.bfloat16, p.T, p.H)
    if saved.numel() < saved_size(p):
        raise MokError(ERR_INVALID, "mok_checkpoint_save: saved")
    rs = routing_struct(routing)
    _check(lib().mok_checkpoint_save(ctypes.byref(p), x.data_ptr(), ctypes.byref(rs), saved.data_ptr(),
                                     ckpt.data_ptr(), ckpt.numel(), _stream(stream)), "mok_checkpoint_save")


def checkpoint_load(p: Problem, ckpt, routing, x, saved, stream=None):
    """x and the saved context, restored for moe_backward."""
    _dense("x", x, torch.bfloat16, p.T, p.H)
    if saved.numel() < saved_size(p):
        raise MokError(ERR_INVALID, "mok_checkpoint_load: saved")
    rs = routing_struct(routing)
    _check(lib().mok_checkpoint_load(ctypes.byref(p), ckpt.data_ptr(), ckpt.numel(), ctypes.byref(rs), x.data_ptr(),
                                     saved.data_ptr(), _stream(stream)), "mok_checkpoint_load")


# --------------------------------------------------------------------------- rows sorted by given experts

BF16_ROWS, F16_ROWS, F32_ROWS = range(3)   # mok_elem
_ELEMS = {torch.bfloat16: BF16_ROWS, torch.float16: F16_ROWS, torch.float32: F32_ROWS}


def _elem(name, t):
    """(mok_elem, device) of a tensor on the current device."""
    elem, dev = _ELEMS.get(t.dtype), t.get_device()
    if elem is None or dev < 0 or dev != torch._C._cuda_getDevice():
        raise AssertionError(f"{name}: bf16, fp16 or fp32 tensor on the current CUDA device expected")
    return elem, dev


class SortLayout(dict):
    """sort_layout's arrays by name, and the tokens and entries per token that they are of."""
    __slots__ = ("tokens", "k")


def sort_workspace_size(T, E, k) -> int:
    return int(lib().mok_sort_workspace_size(T, E, k))


def sort_layout(topk_idx, E, out=None, workspace=None, stream=None):
    """Layout of rows sorted by given expert indices [T, k] int32 (outside 0..E-1: dropped), for sort_rows and
    unsort_rows. With topk_idx and topk_w beside it, it is the layer's routing too where no entry is dropped and no
    token names an expert twice. Returns a SortLayout (a dict) of counts [E], offsets [E+1], row_src [T*k], slot_row [T*k] (see
    mok_sort_layout); new ones are `stream`'s in the allocator."""
    T, k = topk_idx.shape
    dev = topk_idx.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice() or topk_idx.dtype is not torch.int32 or not topk_idx.is_contiguous():
        raise AssertionError("topk_idx: contiguous int32 tensor on the current CUDA device expected")
    n = T * k
    if out is None or workspace is None:
        with _allocating(stream):
            if out is None:
                out = SortLayout((name, torch.empty(size, dtype=torch.int32, device=topk_idx.device))
                                 for name, size in (("counts", E), ("offsets", E + 1), ("row_src", n), ("slot_row", n)))
            if workspace is None:
                workspace = alloc_bytes(sort_workspace_size(T, E, k), topk_idx.device)
    counts, offsets, row_src, slot_row = out["counts"], out["offsets"], out["row_src"], out["slot_row"]
    _here("counts", counts, dev, torch.int32, E)
    _here("offsets", offsets, dev, torch.int32, E + 1)
    _here("row_src", row_src, dev, torch.int32, n)
    _here("slot_row", slot_row, dev, torch.int32, n)
    _check(lib().mok_sort_layout(topk_idx.data_ptr(), T, E, k, counts.data_ptr(), offsets.data_ptr(),
                                 row_src.data_ptr(), slot_row.data_ptr(), _scratch(workspace, dev), workspace.numel(),
                                 _stream(stream)), "mok_sort_layout")
    if out.__class__ is not SortLayout:
        out = SortLayout(out)
    out.tokens = T
    out.k = k
    return out


def _slots(layout, T, device, w=None):
    """(slot_row, k) of a layout of T tokens on this device. Of no tokens, k is the layout's or the weights'."""
    s = layout["slot_row"]
    n = s.numel()
    if layout.__class__ is SortLayout and layout.tokens != T:
        raise AssertionError(f"layout: of {T} tokens expected, not of {layout.tokens}")
    if T <= 0:
        if n or T:
            raise AssertionError("slot_row: of these tokens expected")
        return s, getattr(layout, "k", None) or (w.shape[1] if w is not None and w.dim() == 2 else 1)
    if n % T or n == 0 or ("topk_idx" in layout and layout["topk_idx"].shape[0] != T):
        raise AssertionError(f"layout: of {T} tokens expected")
    _here("slot_row", s, device, torch.int32, n)
    return s, n // T


def sort_rows(x, layout, out, stream=None):
    """Rows of x [T, H] at their entries' places in out [T*k, H]; later rows of out are left as they are.
    unsort_rows without weights is the gradient."""
    T, H = x.shape
    elem, dev = _elem("x", x)
    slot, k = _slots(layout, T, dev)
    pitch, step = x.stride()
    if step != 1 and T:
        raise AssertionError("x: adjacent row elements expected")
    _here("out", out, dev, x.dtype, T * k, H)
    _check(lib().mok_sort_rows(x.data_ptr(), pitch if T > 1 else H, slot.data_ptr(), T, H, k, elem, out.data_ptr(),
                               _stream(stream)), "mok_sort_rows")
    return out


def unsort_rows(y, layout, out, w=None, stream=None):
    """out [T, H] = the sum of each token's rows of y [T*k, H], times w [T, k] (fp32) if given."""
    T, H = out.shape
    elem, dev = _elem("out", out)
    slot, k = _slots(layout, T, dev, w)
    _here("out", out, dev, out.dtype, T, H)
    _here("y", y, dev, out.dtype, T * k, H)
    _here("w", w, dev, torch.float32, T, k)
    _check(lib().mok_unsort_rows(y.data_ptr(), slot.data_ptr(), _addr(w), T, H, k, elem, out.data_ptr(),
                                 _stream(stream)), "mok_unsort_rows")
    return out


def unsort_rows_backward(dout, y, layout, w, dy, dw, stream=None):
    """Gradients of unsort_rows: dy [T*k, H] (later rows are left as they are) and dw [T, k]."""
    T, H = dout.shape
    elem, dev = _elem("dout", dout)
    slot, k = _slots(layout, T, dev, w)
    _here("dout", dout, dev, dout.dtype, T, H)
    _here("y", y, dev, dout.dtype, T * k, H)
    _here("dy", dy, dev, dout.dtype, T * k, H)
    _here("w", w, dev, torch.float32, T, k)
    _here("dw", dw, dev, torch.float32, T, k)
    _check(lib().mok_unsort_rows_backward(dout.data_ptr(), y.data_ptr(), slot.data_ptr(), w.data_ptr(), T, H, k, elem,
                                          dy.data_ptr(), dw.data_ptr(), _stream(stream)), "mok_unsort_rows_backward")


# --------------------------------------------------------------------------- loss of the vocabulary's head

HEAD_DX, HEAD_DW, HEAD_DW_F32 = 2, 4, 8   # MOK_HEAD_*


def head_workspace_size(T, H, V, grad=False, piece=0, cfg: Config | None = None) -> int:
    """grad: False for head_loss, the sum of the HEAD_* gradients that the call forms, or True for any."""
    return int(lib().mok_head_workspace_size(T, H, V, int(grad), piece, ctypes.byref(cfg) if cfg else None))


def _head_args(x, W, labels, workspace, piece, loss=None, lse=None, dloss=None, scale=1.0, dx=None, dW=None,
               accumulate=False):
    T, H = x.shape
    V = W.shape[0]
    pitch = _rows("x", x, T, H)
    dev = x.get_device()
    if dev != torch._C._cuda_getDevice():
        raise AssertionError("x: on the current CUDA device expected")
    _here("W", W, dev, torch.bfloat16, V, H)
    if labels.dtype not in (torch.int32, torch.int64):
        raise AssertionError("labels: int32 or int64 expected")
    _here("labels", labels, dev, labels.dtype, T)
    for n, t in (("loss", loss), ("lse", lse), ("dloss", dloss)):
        _here(n, t, dev, torch.float32, T)
    _here("dx", dx, dev, torch.bfloat16, T, H)
    f32 = dW is not None and dW.dtype is torch.float32
    _here("dW", dW, dev, torch.float32 if f32 else torch.bfloat16, V, H)
    return T, H, V, HeadArgs(x.data_ptr(), pitch, W.data_ptr(), labels.data_ptr(), labels.dtype is torch.int64, piece,
                             _addr(loss), _addr(lse), _addr(dloss), scale, f32, bool(accumulate), _addr(dx), _addr(dW),
                             _scratch(workspace, dev), workspace.numel())


def _head_call(name, a, cfg, stream):
    T, H, V, args = a
    _check(getattr(lib(), name)(T, H, V, ctypes.byref(args), ctypes.byref(cfg) if cfg else None, _stream(stream)), name)


def head_loss(x, W, labels, loss, workspace, lse=None, cfg: Config | None = None, stream=None):
    """Softmax cross entropy of x [T, H] against the vocabulary's rows W [V, H] (see mok_head_loss). labels: int32 or
    int64, outside 0..V-1: ignored. x may be a row-strided view."""
    _head_call("mok_head_loss", _head_args(x, W, labels, workspace, 0, loss, lse), cfg, stream)
    return loss


def head_loss_backward(x, W, labels, lse, dx, dW, workspace, dloss=None, scale=1.0, accumulate=False, piece=0,
                       cfg: Config | None = None, stream=None):
    """Gradients dx [T, H] and dW [V, H] (bf16 or fp32; either may be None) from head_loss's lse, for the losses'
    gradient scale * dloss. accumulate: dW (fp32) is added to."""
    _head_call("mok_head_loss_backward",
               _head_args(x, W, labels, workspace, piece, None, lse, dloss, scale, dx, dW, accumulate), cfg, stream)


def head_loss_train(x, W, labels, loss, dx, dW, workspace, dloss=None, scale=1.0, lse=None, accumulate=False, piece=0,
                    cfg: Config | None = None, stream=None):
    """head_loss and head_loss_backward in one call, for a dloss that does not depend on the loss."""
    _head_call("mok_head_loss_train",
               _head_args(x, W, labels, workspace, piece, loss, lse, dloss, scale, dx, dW, accumulate), cfg, stream)
    return loss


# --------------------------------------------------------------------------- gradient norm and clipping

class GradList:
    """Gradients (and where their clipped values go) in the form the library takes; keeps the tensors."""

    def __init__(self, grads, out=None):
        self.tensors, self.out = list(grads), None if out is None else list(out)
        if self.out is not None and len(self.out) != len(self.tensors):
            raise AssertionError("out: a tensor for each gradient expected")
        n = len(self.tensors)
        self.array, self.count = (GradTensor * max(n, 1))(), n
        spans = []
        for i, g in enumerate(self.tensors):
            (elem, dev), o = _elem(f"grads[{i}]", g), None if self.out is None else self.out[i]
            _here(f"grads[{i}]", g, dev, g.dtype, *g.shape)
            _here(f"out[{i}]", o, dev, g.dtype, *g.shape)
            self.array[i] = GradTensor(g.data_ptr(), _addr(o), g.numel(), elem)
            for t in (g,) if o is None or o.data_ptr() == g.data_ptr() else (g, o):
                if t.numel():
                    spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()))
        spans.sort()
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise AssertionError("gradients and outputs that do not overlap expected")
        self.device = torch._C._cuda_getDevice() if n else None

    def check(self):
        """The current device is the one that the gradients are on."""
        if self.count and self.device != torch._C._cuda_getDevice():
            raise AssertionError("gradients on the current CUDA device expected")
        return self


def grad_list(grads, out=None) -> GradList:
    """Made once for gradients that stay where they are; grad_norm and grad_clip take it in place of a list."""
    return GradList(grads, out)


def grad_workspace_size() -> int:
    return int(lib().mok_grad_workspace_size())


def _norm_device(norm):
    """The current device, on which the norm has to be."""
    dev = norm.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice() or norm.dtype is not torch.float32 or norm.dim():
        raise AssertionError("norm: fp32 tensor [] on the current CUDA device expected")
    return dev


def grad_norm(grads, norm, workspace, stream=None):
    """norm [] (fp32) = 2-norm of all elements of a list of bf16, fp16 and fp32 tensors."""
    g = grads.check() if isinstance(grads, GradList) else GradList(grads)
    _check(lib().mok_grad_norm(g.count, g.array, norm.data_ptr(), _scratch(workspace, _norm_device(norm)),
                               workspace.numel(), _stream(stream)), "mok_grad_norm")
    return norm


def grad_clip(grads, max_norm, norm, workspace, stream=None):
    """norm as grad_norm, and all gradients times min(1, max_norm / (norm + 1e-6)): in place, or into a grad_list's
    outputs."""
    g = grads.check() if isinstance(grads, GradList) else GradList(grads)
    _check(lib().mok_grad_clip(g.count, g.array, float(max_norm), norm.data_ptr(),
                               _scratch(workspace, _norm_device(norm)), workspace.numel(), _stream(stream)),
           "mok_grad_clip")
    return norm


def megakernel_trace(workspace, n_ctas):
    """Per-CTA megakernel records written under FLAG_TRACE: int64 [n_ctas, 8]
    (role, t_begin, t_first, t_work_end, t_exit, wait_ns, units, combine_ns)."""
    return workspace[256:256 + 64 * n_ctas].view(torch.int64).view(n_ctas, 8).cpu().numpy()


def route_test_hook(withhold_copy, timeout_ms=0):
    """Test hook of the routing kernels' bounded waits (see mok.h)."""
    _check(lib().mok_route_test_hook(int(withhold_copy), int(timeout_ms)), "mok_route_test_hook")


def device_status(workspace, reset=False, stream=None):
    """(status code, detail) recorded on the device by the last call; with
    workspace None, the last mok_route_layout_static call on this device."""
    d = ctypes.c_int32(0)
    rc = lib().mok_device_status(_ptr(workspace), _stream(stream), ctypes.byref(d), int(reset))
    return int(rc), int(d.value)


def check_device_status(workspace, what="device", stream=None):
    rc, d = device_status(workspace, stream=stream)
    if rc != OK:
        raise MokError(rc, f"{what} (detail {d})")


# --------------------------------------------------------------------------- expert parallelism

def ep_workspace_size(G, E) -> int:
    return int(lib().mok_ep_workspace_size(G, E))


def _peers(peers):
    arr = (EpPeer * len(peers))()
    for i, q in enumerate(peers):
        arr[i] = EpPeer(q["x"].data_ptr() if q.get("x") is not None else None, q["offsets"].data_ptr(),
                        q["row_src"].data_ptr() if q.get("row_src") is not None else None,
                        q["partials"].data_ptr() if q.get("partials") is not None else None, int(q["T"]))
    return arr


def ep_dispatch(G, rank, H, E, k, peers, counts_all, A, rows_cap, counts_local, offsets_local, src_rank, src_slot,
                ident, workspace, stream=None):
    """peers: list of G dicts {x, offsets, row_src, partials, T} (device tensors)."""
    rc = lib().mok_ep_dispatch(G, rank, H, E, k, _peers(peers), _ptr(counts_all), _ptr(A), int(rows_cap),
                               _ptr(counts_local), _ptr(offsets_local), _ptr(src_rank), _ptr(src_slot), _ptr(ident),
                               _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "mok_ep_dispatch")


def ep_push(G, H, E, k, peers, ys, rows_cap, offsets_local, src_rank, src_slot, stream=None):
    rc = lib().mok_ep_push(G, H, E, k, _peers(peers), _ptr(ys), int(rows_cap), _ptr(offsets_local), _ptr(src_rank),
                           _ptr(src_slot), _stream(stream))
    _check(rc, "mok_ep_push")
