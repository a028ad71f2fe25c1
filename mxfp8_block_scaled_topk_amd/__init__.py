"""Python binding of libmxmoe.so, the MXFP8 block-scaled top-k MoE expert
layer for AMD MI355X (gfx950).

Argument marshalling only: every step runs in the library's HIP kernels.
Tensors are torch tensors on the GPU (torch supplies device memory and the
current stream); outputs are allocated here when not passed in and carry no
autograd graph, whatever the inputs require.  Any non-OK status from the library
raises ``MxError`` with the library's message.

Formats (see include/mxmoe.h): e4m3 payloads and e8m0 scales are uint8
tensors; scales use the pair-split layout [rows, ceil(cols/64), 2]; int8 codes
are torch.int8 with fp32 scales per row; bf16 tensors are torch.bfloat16; group
lists are int64 (type 1 = counts, type 0 = inclusive cumulative counts).
"""

import ctypes
import functools
import inspect
import os

import torch

__all__ = [
    "MxError", "lib_path", "load", "mx_quantize", "moe_route_quant", "gmm_swiglu_mxquant",
    "gmm_mx", "moe_finalize", "moe_mxfp8_forward", "forward_workspace", "forward_intermediates",
    "route_workspace_size", "forward_workspace_size", "last_error", "moe_router", "mx_linear",
    "linear_workspace_size", "mx_quantize_fp4", "moe_route_quant_noalloc", "mx_pack_weights", "route_set_wait_limit",
    "gmm_swiglu_mxquant_packed", "gmm_mx_packed", "moe_mxfp8_forward_packed", "gmm_mx_w4a8", "gmm_swiglu_mxquant_w4a8", "moe_w4a8_forward",
    "mx_linear_fused", "linear_fused_workspace_size", "linear_fused_kernel", "mx_add_rmsnorm", "moe_route_mx", "moe_mxfp8_forward_mx",
    "int8_quantize", "int8_linear", "int8_linear_workspace_size", "int8_linear_kernel", "gmm_int8", "gmm_int8_kernel", "moe_permute", "moe_unpermute",
    "moe_unpermute_backward",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

MX_OK = 0
GROUP_CUMULATIVE = 0
GROUP_COUNT = 1


class MxError(RuntimeError):
    """A non-OK status from libmxmoe."""


def lib_path():
    return os.path.join(_HERE, "libmxmoe.so")


def load():
    """Load libmxmoe.so (built by ``python -m mxfp8_block_scaled_topk_amd.build``).

    There is no fallback: a missing library is an error."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise MxError(f"{path} is missing; build it with `python -m mxfp8_block_scaled_topk_amd.build`")
    lib = ctypes.CDLL(path)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sig = {
        "mx_quantize": (I32, [P, I64, I64, I64, P, P, P]),
        "mx_quantize_fp4": (I32, [P, I64, I64, I64, P, P, P]),
        "moe_route_quant_workspace_size": (SZ, [I64, I64, I64]),
        "moe_route_quant": (I32, [P, P, I64, I64, I64, I64, P, P, P, P, P, P, SZ, P]),
        "moe_route_quant_noalloc": (I32, [P, P, I64, I64, I64, I64, P, P, P, P, P, P]),
        "moe_route_quant_set_wait_limit": (I64, [I64]),
        "gmm_swiglu_mxquant": (I32, [P, P, P, P, P, I32, I64, I64, I64, I64, P, P, P, P]),
        "gmm_mx": (I32, [P, P, P, P, P, I32, I64, I64, I64, I64, P, P]),
        "gmm_mx_w4a8": (I32, [P, P, P, P, P, I32, I64, I64, I64, I64, P, P]),
        "gmm_swiglu_mxquant_w4a8": (I32, [P, P, P, P, P, I32, I64, I64, I64, I64, P, P, P, P]),
        "moe_w4a8_forward": (I32, [P, P, P, P, P, P, P, I64, I64, I64, I64, I64, P, P, SZ, P]),
        "moe_finalize": (I32, [P, P, P, I64, I64, I64, I64, P, P]),
        "moe_mxfp8_forward_workspace_size": (SZ, [I64, I64, I64, I64, I64]),
        "moe_mxfp8_forward": (I32, [P, P, P, P, P, P, P, I64, I64, I64, I64, I64, P, P, SZ, P]),
        "moe_mxfp8_forward_workspace_layout": (I32, [I64, I64, I64, I64, I64, P]),
        "moe_router": (I32, [P, P, P, I64, I64, I64, I64, I32, P, P, P]),
        "mx_linear_workspace_size": (SZ, [I64, I64]),
        "mx_linear": (I32, [P, P, P, I64, I64, I64, P, P, SZ, P]),
        "mx_pack_weights": (I32, [P, I64, I64, I64, I32, P, P]),
        "gmm_swiglu_mxquant_packed": (I32, [P, P, P, P, P, I32, I64, I64, I64, I64, P, P, P, P]),
        "gmm_mx_packed": (I32, [P, P, P, P, P, I32, I64, I64, I64, I64, P, P]),
        "moe_mxfp8_forward_packed": (I32, [P, P, P, P, P, P, P, I64, I64, I64, I64, I64, P, P, SZ, P]),
        "mx_add_rmsnorm": (I32, [P, I64, P, I64, P, I32, ctypes.c_float, I64, I64, P, P, P, P, P]),
        "moe_route_mx": (I32, [P, P, P, I64, I64, I64, I64, P, P, P, P, P, P, SZ, P]),
        "moe_mxfp8_forward_mx": (I32, [P, P, P, P, I32, P, P, P, P, I64, I64, I64, I64, I64, P, P, SZ, P]),
        "mx_linear_fused_workspace_size": (SZ, [I64, I64, I64, I32]),
        "mx_linear_fused_kernel": (I32, [I64, I64, I64, I32]),
        "mx_linear_fused": (I32, [P, P, P, P, P, I32, I32, P, I64, I64, I64, P, P, P, P, SZ, P]),
        "int8_quantize": (I32, [P, I64, I64, I64, P, P, P]),
        "int8_linear_workspace_size": (SZ, [I64, I64, I64, I32]),
        "int8_linear": (I32, [P, P, P, P, P, I32, I32, P, I64, I64, I64, P, P, SZ, P]),
        "int8_linear_kernel": (I32, [I64, I64, I64, I32]),
        "gmm_int8_kernel": (I32, [I64, I64, I64, I64, I32]),
        "gmm_int8": (I32, [P, P, P, P, P, I32, I32, I64, I64, I64, I64, P, P]),
        "moe_permute": (I32, [P, I64, I64, P, P, I64, I64, I64, I64, P, P, P, P, P, P, SZ, P]),
        "moe_unpermute": (I32, [P, I32, P, P, I64, I64, I64, I64, P, P]),
        "moe_unpermute_backward": (I32, [P, I32, P, P, P, I64, I64, I64, I64, P, P, P]),
        "mx_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _LIB = lib
    return lib


def last_error():
    return load().mx_last_error().decode()


def _check(rc, what):
    if rc != MX_OK:
        raise MxError(f"{what}: status {rc}: {last_error()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _stream_scoped(fn):
    """Run ``fn`` with its ``stream`` argument (when given) as torch's current
    stream.  Every tensor the binding allocates for the call (outputs left to
    it, internal workspaces) then comes from that stream's pool of the caching
    allocator: freed on return, such a workspace is reused only by later work
    on the same stream, which runs after the kernels that used it.  Allocated
    on another stream instead, it could be handed to work on that stream while
    the kernels still read or write it."""
    sig = inspect.signature(fn)

    @functools.wraps(fn)
    def wrapper(*args, **kw):
        s = sig.bind(*args, **kw).arguments.get("stream")
        if s is None:
            return fn(*args, **kw)
        with torch.cuda.stream(s):
            return fn(*args, **kw)
    return wrapper


# Argument checks.  The library receives raw pointers and sizes, so every
# tensor is checked here for dtype, exact shape, contiguity and device before
# the call: a tensor smaller than its sizes say would be read or written out
# of bounds on the GPU.  Shape checks come first and residency on the GPU
# last, so that shape errors are reported the same way on any device.

def _need(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _need_shape(t, shape, name, dtype, device):
    """t: a contiguous `dtype` tensor of exactly `shape` on `device`."""
    _need(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _need_workspace(ws, nbytes, device, name="workspace"):
    _need(ws, torch.uint8, name, 1)
    if not ws.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ws.device != device:
        raise ValueError(f"{name} must be on {device}, got {ws.device}")
    if ws.numel() < nbytes:
        raise ValueError(f"{name} has {ws.numel()} bytes, {nbytes} needed")


def _need_gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")


def _pairs(n):
    return -(-n // 64)


@_stream_scoped
def mx_quantize(x, q=None, s=None, stream=None):
    """MX-quantise the last dim of a bf16 tensor [..., Kd] (rows may be strided
    with unit inner stride).  Returns (q uint8 [..., Kd], s uint8 [..., ceil(Kd/64), 2])."""
    _need(x, torch.bfloat16, "x")
    kd = x.shape[-1]
    lead = tuple(x.shape[:-1])
    x2 = x.reshape(-1, kd) if x.dim() != 2 else x
    if x2.stride(-1) != 1:
        raise ValueError("x must have unit stride along the last dim")
    rows = x2.shape[0]
    if q is None:
        q = torch.empty(lead + (kd,), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty(lead + (_pairs(kd), 2), dtype=torch.uint8, device=x.device)
    _need_shape(q, lead + (kd,), "q", torch.uint8, x.device)
    _need_shape(s, lead + (_pairs(kd), 2), "s", torch.uint8, x.device)
    ld = x2.stride(0) if rows > 1 else kd
    _need_gpu(x, "x")
    rc = load().mx_quantize(_ptr(x2), rows, kd, ld, _ptr(q), _ptr(s), _stream(stream))
    _check(rc, "mx_quantize")
    return q, s


def route_workspace_size(T, k, E):
    return int(load().moe_route_quant_workspace_size(T, k, E))


def route_set_wait_limit(polls):
    """Polls a routing workgroup makes for the published expert counts before
    counting them itself (process-wide; 0 = always count). Returns the
    previous value."""
    return int(load().moe_route_quant_set_wait_limit(int(polls)))


@_stream_scoped
def moe_route_quant(x, topk_ids, E, out=None, workspace=None, stream=None):
    """Routing with fused MX activation quant.

    Returns (xq [M,K] u8, xs [M,K/64,2] u8, sorted_row [M] i32,
    expanded_row_idx [M] i32, group_list [E] i64 counts)."""
    _need(x, torch.bfloat16, "x", 2); _need(topk_ids, torch.int32, "topk_ids", 2)
    T, K = x.shape
    k = topk_ids.shape[1]
    M = T * k
    dev = x.device
    _need_shape(x, (T, K), "x", torch.bfloat16, dev)
    _need_shape(topk_ids, (T, k), "topk_ids", torch.int32, dev)
    if out is None:
        out = (torch.empty((M, K), dtype=torch.uint8, device=dev),
               torch.empty((M, _pairs(K), 2), dtype=torch.uint8, device=dev),
               torch.empty(M, dtype=torch.int32, device=dev),
               torch.empty(M, dtype=torch.int32, device=dev),
               torch.empty(E, dtype=torch.int64, device=dev))
    xq, xs, sr, eri, gl = out
    _need_shape(xq, (M, K), "xq", torch.uint8, dev)
    _need_shape(xs, (M, _pairs(K), 2), "xs", torch.uint8, dev)
    _need_shape(sr, (M,), "sorted_row", torch.int32, dev)
    _need_shape(eri, (M,), "expanded_row_idx", torch.int32, dev)
    _need_shape(gl, (E,), "group_list", torch.int64, dev)
    need = route_workspace_size(T, k, E)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _need_workspace(workspace, need, dev)
    _need_gpu(x, "x")
    rc = load().moe_route_quant(_ptr(x), _ptr(topk_ids), T, K, k, E, _ptr(xq), _ptr(xs), _ptr(sr), _ptr(eri),
                                _ptr(gl), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "moe_route_quant")
    return xq, xs, sr, eri, gl


@_stream_scoped
def moe_route_quant_noalloc(x, topk_ids, E, out=None, stream=None):
    """moe_route_quant with the routing scratch held by the library (no
    workspace; the C call allocates nothing).  The caller may pass the
    outputs preallocated in ``out`` (then this call allocates nothing either).
    Returns (xq, xs, sorted_row, expanded_row_idx, group_list)."""
    _need(x, torch.bfloat16, "x", 2); _need(topk_ids, torch.int32, "topk_ids", 2)
    T, K = x.shape
    k = topk_ids.shape[1]
    M = T * k
    dev = x.device
    _need_shape(x, (T, K), "x", torch.bfloat16, dev)
    _need_shape(topk_ids, (T, k), "topk_ids", torch.int32, dev)
    if out is None:
        out = (torch.empty((M, K), dtype=torch.uint8, device=dev),
               torch.empty((M, _pairs(K), 2), dtype=torch.uint8, device=dev),
               torch.empty(M, dtype=torch.int32, device=dev),
               torch.empty(M, dtype=torch.int32, device=dev),
               torch.empty(E, dtype=torch.int64, device=dev))
    xq, xs, sr, eri, gl = out
    _need_shape(xq, (M, K), "xq", torch.uint8, dev)
    _need_shape(xs, (M, _pairs(K), 2), "xs", torch.uint8, dev)
    _need_shape(sr, (M,), "sorted_row", torch.int32, dev)
    _need_shape(eri, (M,), "expanded_row_idx", torch.int32, dev)
    _need_shape(gl, (E,), "group_list", torch.int64, dev)
    _need_gpu(x, "x")
    rc = load().moe_route_quant_noalloc(_ptr(x), _ptr(topk_ids), T, K, k, E, _ptr(xq), _ptr(xs), _ptr(sr), _ptr(eri),
                                        _ptr(gl), _stream(stream))
    _check(rc, "moe_route_quant_noalloc")
    return xq, xs, sr, eri, gl


@_stream_scoped
def gmm_swiglu_mxquant(a, a_s, w13, w13_s, group_list, group_list_type=GROUP_COUNT, out=None,
                       h_debug=False, stream=None, _w4=False, _packed=False):
    """GEMM1 + SwiGLU + MX requant.  Returns (hq, hs) or (hq, hs, h) with h_debug."""
    _need(a, torch.uint8, "a", 2); _need(w13, torch.uint8, "w13", 3)
    M, K = a.shape
    E, twoI, Kw = w13.shape
    Kb = K // 2 if _w4 else K           # weight payload bytes per row
    if Kw != Kb or twoI % 2:
        raise ValueError(f"w13 must be [E, 2I, {Kb}], got {tuple(w13.shape)}")
    I = twoI // 2
    dev = a.device
    _need_shape(a, (M, K), "a", torch.uint8, dev)
    _need_shape(a_s, (M, _pairs(K), 2), "a_s", torch.uint8, dev)
    _need_shape(w13, (E, twoI, Kb), "w13", torch.uint8, dev)
    _need_shape(w13_s, (E, twoI, _pairs(K), 2), "w13_s", torch.uint8, dev)
    _need_shape(group_list, (E,), "group_list", torch.int64, dev)
    if out is None:
        out = (torch.empty((M, I), dtype=torch.uint8, device=dev),
               torch.empty((M, _pairs(I), 2), dtype=torch.uint8, device=dev))
    hq, hs = out
    _need_shape(hq, (M, I), "hq", torch.uint8, dev)
    _need_shape(hs, (M, _pairs(I), 2), "hs", torch.uint8, dev)
    h = torch.empty((M, I), dtype=torch.float32, device=dev) if h_debug else None
    _need_gpu(a, "a")
    name = "gmm_swiglu_mxquant_w4a8" if _w4 else "gmm_swiglu_mxquant_packed" if _packed else "gmm_swiglu_mxquant"
    rc = getattr(load(), name)(_ptr(a), _ptr(a_s), _ptr(w13), _ptr(w13_s), _ptr(group_list), group_list_type, M, K,
                               I, E, _ptr(hq), _ptr(hs), _ptr(h), _stream(stream))
    _check(rc, name)
    return (hq, hs, h) if h_debug else (hq, hs)


@_stream_scoped
def gmm_mx(a, a_s, w, w_s, group_list, group_list_type=GROUP_COUNT, out=None, stream=None, _w4=False,
           _packed=False):
    """Grouped MX GEMM, bf16 output [M, N]."""
    _need(a, torch.uint8, "a", 2); _need(w, torch.uint8, "w", 3)
    M, Kd = a.shape
    E, N, Kw = w.shape
    Kb = Kd // 2 if _w4 else Kd
    if Kw != Kb:
        raise ValueError(f"w must be [E, N, {Kb}], got {tuple(w.shape)}")
    dev = a.device
    _need_shape(a, (M, Kd), "a", torch.uint8, dev)
    _need_shape(a_s, (M, _pairs(Kd), 2), "a_s", torch.uint8, dev)
    _need_shape(w, (E, N, Kb), "w", torch.uint8, dev)
    _need_shape(w_s, (E, N, _pairs(Kd), 2), "w_s", torch.uint8, dev)
    _need_shape(group_list, (E,), "group_list", torch.int64, dev)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _need_shape(out, (M, N), "out", torch.bfloat16, dev)
    _need_gpu(a, "a")
    name = "gmm_mx_w4a8" if _w4 else "gmm_mx_packed" if _packed else "gmm_mx"
    rc = getattr(load(), name)(_ptr(a), _ptr(a_s), _ptr(w), _ptr(w_s), _ptr(group_list), group_list_type, M, N, Kd,
                               E, _ptr(out), _stream(stream))
    _check(rc, name)
    return out


@_stream_scoped
def moe_finalize(y, topk_w, expanded_row_idx, out=None, stream=None):
    """Weighted un-permute and sum: out [T, K] bf16."""
    _need(y, torch.bfloat16, "y", 2); _need(topk_w, torch.float32, "topk_w", 2)
    _need(expanded_row_idx, torch.int32, "expanded_row_idx")
    M, K = y.shape
    T, k = topk_w.shape
    dev = y.device
    _need_shape(y, (M, K), "y", torch.bfloat16, dev)
    _need_shape(topk_w, (T, k), "topk_w", torch.float32, dev)
    if expanded_row_idx.numel() != T * k:
        raise ValueError(f"expanded_row_idx must hold T*k = {T * k} entries, got {expanded_row_idx.numel()}")
    _need_shape(expanded_row_idx, tuple(expanded_row_idx.shape), "expanded_row_idx", torch.int32, dev)
    if out is None:
        out = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
    _need_shape(out, (T, K), "out", torch.bfloat16, dev)
    _need_gpu(y, "y")
    rc = load().moe_finalize(_ptr(y), _ptr(topk_w), _ptr(expanded_row_idx), T, K, k, M, _ptr(out),
                             _stream(stream))
    _check(rc, "moe_finalize")
    return out


def forward_workspace_size(T, K, I, E, k):
    return int(load().moe_mxfp8_forward_workspace_size(T, K, I, E, k))


def forward_workspace(T, K, I, E, k, device="cuda"):
    return torch.empty(max(forward_workspace_size(T, K, I, E, k), 256), dtype=torch.uint8, device=device)


@_stream_scoped
def moe_mxfp8_forward(x, topk_ids, topk_w, w13, w13_s, w2, w2_s, out=None, workspace=None, stream=None,
                      _w4=False, _packed=False):
    """The whole layer.  x [T,K] bf16, topk_ids [T,k] i32, topk_w [T,k] f32,
    w13 [E,2I,K] u8 + w13_s [E,2I,K/64,2], w2 [E,K,I] u8 + w2_s [E,K,I/64,2].
    Returns out [T,K] bf16."""
    _need(x, torch.bfloat16, "x", 2); _need(topk_ids, torch.int32, "topk_ids", 2)
    _need(w13, torch.uint8, "w13", 3)
    T, K = x.shape
    k = topk_ids.shape[1]
    E, twoI, Kw = w13.shape
    Kb = K // 2 if _w4 else K
    if Kw != Kb or twoI % 2:
        raise ValueError(f"w13 must be [E, 2I, {Kb}], got {tuple(w13.shape)}")
    I = twoI // 2
    dev = x.device
    _need_shape(x, (T, K), "x", torch.bfloat16, dev)
    _need_shape(topk_ids, (T, k), "topk_ids", torch.int32, dev)
    _need_shape(topk_w, (T, k), "topk_w", torch.float32, dev)
    _need_shape(w13, (E, twoI, Kb), "w13", torch.uint8, dev)
    _need_shape(w13_s, (E, twoI, _pairs(K), 2), "w13_s", torch.uint8, dev)
    _need_shape(w2, (E, K, I // 2 if _w4 else I), "w2", torch.uint8, dev)
    _need_shape(w2_s, (E, K, _pairs(I), 2), "w2_s", torch.uint8, dev)
    if out is None:
        out = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
    _need_shape(out, (T, K), "out", torch.bfloat16, dev)
    need = forward_workspace_size(T, K, I, E, k)
    if workspace is None:
        workspace = forward_workspace(T, K, I, E, k, dev)
    _need_workspace(workspace, need, dev)
    _need_gpu(x, "x")
    name = "moe_w4a8_forward" if _w4 else "moe_mxfp8_forward_packed" if _packed else "moe_mxfp8_forward"
    rc = getattr(load(), name)(_ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13), _ptr(w13_s), _ptr(w2), _ptr(w2_s),
                               T, K, I, E, k, _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, name)
    return out


def forward_intermediates(workspace, T, K, I, E, k):
    """Views of the intermediates a forward call left in its workspace:
    dict(xq, xs, sorted_row, expanded_row_idx, group_list, hq, hs, y)."""
    offs = (ctypes.c_size_t * 8)()
    _check(load().moe_mxfp8_forward_workspace_layout(T, K, I, E, k, offs), "workspace_layout")
    M = T * k

    def view(i, n, dtype):
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return workspace[offs[i]:offs[i] + nbytes].view(dtype)

    return dict(
        xq=view(0, M * K, torch.uint8).view(M, K),
        xs=view(1, M * _pairs(K) * 2, torch.uint8).view(M, _pairs(K), 2),
        sorted_row=view(2, M, torch.int32),
        expanded_row_idx=view(3, M, torch.int32),
        group_list=view(4, E, torch.int64),
        hq=view(5, M * I, torch.uint8).view(M, I),
        hs=view(6, M * _pairs(I) * 2, torch.uint8).view(M, _pairs(I), 2),
        y=view(7, M * K, torch.bfloat16).view(M, K),
    )


@_stream_scoped
def moe_router(x, gate, k, bias=None, renormalize=True, out=None, stream=None):
    """Top-k softmax router: x [T,K] bf16, gate [E,K] bf16, optional bias [E]
    fp32.  Returns (topk_ids [T,k] int32, topk_w [T,k] float32)."""
    _need(x, torch.bfloat16, "x", 2); _need(gate, torch.bfloat16, "gate", 2)
    T, K = x.shape
    E = gate.shape[0]
    dev = x.device
    _need_shape(x, (T, K), "x", torch.bfloat16, dev)
    _need_shape(gate, (E, K), "gate", torch.bfloat16, dev)
    if bias is not None:
        _need_shape(bias, (E,), "bias", torch.float32, dev)
    if out is None:
        out = (torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), dtype=torch.float32, device=dev))
    ids, w = out
    _need_shape(ids, (T, k), "topk_ids", torch.int32, dev)
    _need_shape(w, (T, k), "topk_w", torch.float32, dev)
    _need_gpu(x, "x")
    rc = load().moe_router(_ptr(x), _ptr(gate), _ptr(bias), T, K, E, k, 1 if renormalize else 0, _ptr(ids), _ptr(w),
                           _stream(stream))
    _check(rc, "moe_router")
    return ids, w


def linear_workspace_size(T, K):
    return int(load().mx_linear_workspace_size(T, K))


@_stream_scoped
def mx_linear(x, w, w_s, out=None, workspace=None, stream=None):
    """Dense MXFP8 linear: x [T,K] bf16, w [N,K] e4m3 bytes, w_s [N,K/64,2]
    e8m0 bytes (as mx_quantize makes them).  Returns y [T,N] bf16."""
    _need(x, torch.bfloat16, "x", 2); _need(w, torch.uint8, "w", 2)
    T, K = x.shape
    N = w.shape[0]
    dev = x.device
    _need_shape(x, (T, K), "x", torch.bfloat16, dev)
    _need_shape(w, (N, K), "w", torch.uint8, dev)
    _need_shape(w_s, (N, _pairs(K), 2), "w_s", torch.uint8, dev)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    _need_shape(out, (T, N), "out", torch.bfloat16, dev)
    need = linear_workspace_size(T, K)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _need_workspace(workspace, need, dev)
    _need_gpu(x, "x")
    if workspace.data_ptr() % 256:
        raise ValueError("workspace must be 256-byte aligned")
    rc = load().mx_linear(_ptr(x), _ptr(w), _ptr(w_s), T, K, N, _ptr(out), _ptr(workspace), workspace.numel(),
                          _stream(stream))
    _check(rc, "mx_linear")
    return out


@_stream_scoped
def mx_quantize_fp4(x, q=None, s=None, stream=None):
    """MXFP4-quantise the last dim of a bf16 tensor [..., Kd] (Kd % 32 == 0).
    Returns (q uint8 [..., Kd/2] packed e2m1, s uint8 [..., ceil(Kd/64), 2])."""
    _need(x, torch.bfloat16, "x")
    kd = x.shape[-1]
    lead = tuple(x.shape[:-1])
    x2 = x.reshape(-1, kd) if x.dim() != 2 else x
    if x2.stride(-1) != 1:
        raise ValueError("x must have unit stride along the last dim")
    if kd % 2:
        raise ValueError("Kd must be even (two codes per byte)")
    rows = x2.shape[0]
    if q is None:
        q = torch.empty(lead + (kd // 2,), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty(lead + (_pairs(kd), 2), dtype=torch.uint8, device=x.device)
    _need_shape(q, lead + (kd // 2,), "q", torch.uint8, x.device)
    _need_shape(s, lead + (_pairs(kd), 2), "s", torch.uint8, x.device)
    ld = x2.stride(0) if rows > 1 else kd
    _need_gpu(x, "x")
    rc = load().mx_quantize_fp4(_ptr(x2), rows, kd, ld, _ptr(q), _ptr(s), _stream(stream))
    _check(rc, "mx_quantize_fp4")
    return q, s


@_stream_scoped
def gmm_swiglu_mxquant_w4a8(a, a_s, w13, w13_s, group_list, group_list_type=GROUP_COUNT, out=None,
                            h_debug=False, stream=None):
    """GEMM1 + SwiGLU + MX requant with MXFP4 weights: w13 [E, 2I, K/2] packed
    e2m1 + w13_s [E, 2I, K/64, 2].  Returns (hq, hs) (MXFP8) or (hq, hs, h)."""
    return gmm_swiglu_mxquant(a, a_s, w13, w13_s, group_list, group_list_type, out, h_debug, stream, _w4=True)


@_stream_scoped
def gmm_mx_w4a8(a, a_s, w, w_s, group_list, group_list_type=GROUP_COUNT, out=None, stream=None):
    """Grouped MX GEMM with MXFP4 weights (w [E, N, Kd/2] packed e2m1), bf16 [M, N]."""
    return gmm_mx(a, a_s, w, w_s, group_list, group_list_type, out, stream, _w4=True)


@_stream_scoped
def moe_w4a8_forward(x, topk_ids, topk_w, w13, w13_s, w2, w2_s, out=None, workspace=None, stream=None):
    """The layer with MXFP4 expert weights: w13 [E,2I,K/2], w2 [E,K,I/2] packed e2m1."""
    return moe_mxfp8_forward(x, topk_ids, topk_w, w13, w13_s, w2, w2_s, out, workspace, stream, _w4=True)


PACK_GEMM2 = 0   # mx_pack_weights kind: plain weight rows (w2, the dense linear)
PACK_GEMM1 = 1   # mx_pack_weights kind: w13, gate rows then up rows


@_stream_scoped
def mx_pack_weights(w, kind, out=None, stream=None):
    """e4m3 expert weights w [E, N, Kd] uint8 -> the tile-packed layout the
    *_packed GEMMs read (same shape and size; see include/mxmoe.h).
    kind: PACK_GEMM1 for w13 [E, 2I, K], PACK_GEMM2 for w2 [E, K, I]."""
    _need(w, torch.uint8, "w", 3)
    E, N, Kd = w.shape
    if out is None:
        out = torch.empty_like(w)
    _need_shape(w, (E, N, Kd), "w", torch.uint8, w.device)
    _need_shape(out, (E, N, Kd), "out", torch.uint8, w.device)
    _need_gpu(w, "w")
    rc = load().mx_pack_weights(_ptr(w), E, N, Kd, int(kind), _ptr(out), _stream(stream))
    _check(rc, "mx_pack_weights")
    return out


def gmm_swiglu_mxquant_packed(a, a_s, w13_packed, w13_s, group_list, group_list_type=GROUP_COUNT, out=None,
                              h_debug=False, stream=None):
    """gmm_swiglu_mxquant with w13 tile-packed (mx_pack_weights, PACK_GEMM1)."""
    return gmm_swiglu_mxquant(a, a_s, w13_packed, w13_s, group_list, group_list_type, out, h_debug, stream,
                              _packed=True)


def gmm_mx_packed(a, a_s, w_packed, w_s, group_list, group_list_type=GROUP_COUNT, out=None, stream=None):
    """gmm_mx with w tile-packed (mx_pack_weights, PACK_GEMM2)."""
    return gmm_mx(a, a_s, w_packed, w_s, group_list, group_list_type, out, stream, _packed=True)


def moe_mxfp8_forward_packed(x, topk_ids, topk_w, w13_packed, w13_s, w2_packed, w2_s, out=None, workspace=None,
                             stream=None):
    """moe_mxfp8_forward with w13 and w2 tile-packed by mx_pack_weights."""
    return moe_mxfp8_forward(x, topk_ids, topk_w, w13_packed, w13_s, w2_packed, w2_s, out, workspace, stream,
                             _packed=True)


# The operators below are called once per layer and decode step, so their
# per-call work on the host is kept small: one pass over the arguments whose
# slow, explaining branch runs only for a wrong one (together about 6 us a call
# less than the checks above).  They run on the device of their first tensor
# whichever device is current.

TYPE_BF16 = 0
TYPE_F32 = 1

# the current stream's handle on a device, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
# the current device's index; only called once a tensor is known to be on a GPU
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_Tensor, _U8, _BF16, _F32 = torch.Tensor, torch.uint8, torch.bfloat16, torch.float32   # (quicker names)


def _need_like(t, shape, name, dtype, device):
    """_need_shape, quick for a right tensor."""
    if not (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device):
        _need_shape(t, shape, name, dtype, device)


def _elsewhere(device, stream):
    """The context a call has to run in: None when `device` is current and no
    stream is given.  With a stream, what the call allocates comes from that
    stream's pool (see _stream_scoped)."""
    if stream is None:
        return None if device.index == _current_device() else torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _addr(t):
    return None if t is None else t.data_ptr()


def _rows(t, name):
    """t [..., K] as (a 2-D view or copy, row stride) with unit inner stride."""
    if t.dim() == 2 and t.is_contiguous():
        return t, t.shape[1]
    t2 = t if t.dim() == 2 else t.reshape(-1, t.shape[-1])
    rows, k = t2.shape
    if k > 1 and t2.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along the last dim")
    ld = t2.stride(0) if rows > 1 else k
    if ld < k:
        raise ValueError(f"{name} must not repeat its rows (row stride {ld} < {k})")
    return t2, ld


def mx_add_rmsnorm(x, weight, residual=None, eps=1e-6, quantize=True, norm_out=False, out=None, stream=None):
    """Residual addition, RMSNorm and MX quantisation of the last dim, one pass:
    h = x + residual, n = h / sqrt(mean(h^2) + eps) * weight in fp32.

    x, residual: bf16 [..., K] (rows may be strided); weight: bf16 or fp32 [K].
    Returns (q, s, residual_out, y): the MXFP8 of n (uint8 [..., K] and
    [..., ceil(K/64), 2]; None without ``quantize``), bf16(h) (None without a
    residual) and bf16(n) (None without ``norm_out``).  ``out`` gives the four
    buffers instead, None for an output that is not wanted; its residual_out
    or y may be x or residual itself."""
    if type(x) is not _Tensor or x.dtype is not _BF16:
        _need(x, _BF16, "x")
    shape, dev = x.shape, x.device
    on_gpu = x.is_cuda
    if on_gpu:   # before _rows, whose copy of strided leading dims belongs to the stream of the call
        there = _elsewhere(dev, stream)
        if there is not None:
            with there:
                return mx_add_rmsnorm(x, weight, residual, eps, quantize, norm_out, out)
    if not shape or shape[-1] == 0:
        raise ValueError("x must have at least one element per row")
    K = shape[-1]
    x2, ldx = _rows(x, "x")
    r2, ldr = None, 0
    if residual is not None:
        if type(residual) is not _Tensor or residual.dtype is not _BF16:
            _need(residual, _BF16, "residual")
        if residual.shape != shape:
            raise ValueError(f"residual must have shape {tuple(shape)}, got {tuple(residual.shape)}")
        if residual.device != dev:
            raise ValueError(f"residual must be on {dev}, got {residual.device}")
        r2, ldr = _rows(residual, "residual")
    wtype = TYPE_F32 if isinstance(weight, _Tensor) and weight.dtype is _F32 else TYPE_BF16
    _need_like(weight, (K,), "weight", _F32 if wtype else _BF16, dev)
    s_shape = (*shape[:-1], -(-K // 64), 2)
    if out is not None:
        q, s, r_out, y = out
        if q is not None:
            _need_like(q, shape, "q", _U8, dev)
        if s is not None:
            _need_like(s, s_shape, "s", _U8, dev)
        if r_out is not None:
            _need_like(r_out, shape, "residual_out", _BF16, dev)
        if y is not None:
            _need_like(y, shape, "y", _BF16, dev)
    if not on_gpu:
        _need_gpu(x, "x")
    if out is None:
        q = torch.empty(shape, dtype=_U8, device=dev) if quantize else None
        s = torch.empty(s_shape, dtype=_U8, device=dev) if quantize else None
        r_out = torch.empty(shape, dtype=_BF16, device=dev) if residual is not None else None
        y = torch.empty(shape, dtype=_BF16, device=dev) if norm_out else None
    rc = load().mx_add_rmsnorm(x2.data_ptr(), ldx, _addr(r2), ldr, weight.data_ptr(), wtype, eps, x2.shape[0], K,
                               _addr(r_out), _addr(y), _addr(q), _addr(s), _raw_stream(dev.index))
    if rc:
        _check(rc, "mx_add_rmsnorm")
    return q, s, r_out, y


def moe_route_mx(q, s, topk_ids, E, out=None, workspace=None, stream=None):
    """moe_route_quant for rows that are MXFP8 already: q uint8 [T, K] and
    s uint8 [T, K/64, 2] (as mx_add_rmsnorm or mx_quantize make them).
    Returns (xq, xs, sorted_row, expanded_row_idx, group_list)."""
    _need(q, _U8, "q", 2)
    if type(topk_ids) is not _Tensor or topk_ids.dim() != 2:
        _need(topk_ids, torch.int32, "topk_ids", 2)
    T, K = q.shape
    k = topk_ids.shape[1]
    M = T * k
    dev = q.device
    P = _pairs(K)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    _need_like(s, (T, P, 2), "s", _U8, dev)
    _need_like(topk_ids, (T, k), "topk_ids", torch.int32, dev)
    if out is not None:
        xq, xs, sr, eri, gl = out
        _need_like(xq, (M, K), "xq", _U8, dev)
        _need_like(xs, (M, P, 2), "xs", _U8, dev)
        _need_like(sr, (M,), "sorted_row", torch.int32, dev)
        _need_like(eri, (M,), "expanded_row_idx", torch.int32, dev)
        _need_like(gl, (E,), "group_list", torch.int64, dev)
    lib = load()
    need = lib.moe_route_quant_workspace_size(T, k, E)
    if workspace is not None:
        _need_workspace(workspace, need, dev)
    _need_gpu(q, "q")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return moe_route_mx(q, s, topk_ids, E, out, workspace)
    if out is None:
        xq = torch.empty((M, K), dtype=_U8, device=dev)
        xs = torch.empty((M, P, 2), dtype=_U8, device=dev)
        sr = torch.empty(M, dtype=torch.int32, device=dev)
        eri = torch.empty(M, dtype=torch.int32, device=dev)
        gl = torch.empty(E, dtype=torch.int64, device=dev)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=_U8, device=dev)
    rc = lib.moe_route_mx(q.data_ptr(), s.data_ptr(), topk_ids.data_ptr(), T, K, k, E, xq.data_ptr(), xs.data_ptr(),
                          sr.data_ptr(), eri.data_ptr(), gl.data_ptr(), _addr(workspace),
                          0 if workspace is None else workspace.numel(), _raw_stream(dev.index))
    if rc:
        _check(rc, "moe_route_mx")
    return xq, xs, sr, eri, gl


WEIGHTS_E4M3 = 0     # e4m3 rows
WEIGHTS_E2M1 = 1     # packed e2m1 (mx_quantize_fp4)
WEIGHTS_PACKED = 2   # e4m3, tile-packed (mx_pack_weights)


def moe_mxfp8_forward_mx(q, s, topk_ids, topk_w, w13, w13_s, w2, w2_s, weight_format=WEIGHTS_E4M3, out=None,
                         workspace=None, stream=None):
    """The whole layer on token rows that are MXFP8 already (q uint8 [T, K],
    s uint8 [T, K/64, 2]); weights as moe_mxfp8_forward, moe_w4a8_forward or
    moe_mxfp8_forward_packed take them, by ``weight_format``.  Returns out
    [T, K] bf16."""
    _need(q, torch.uint8, "q", 2); _need(topk_ids, torch.int32, "topk_ids", 2)
    _need(w13, torch.uint8, "w13", 3)
    if weight_format not in (WEIGHTS_E4M3, WEIGHTS_E2M1, WEIGHTS_PACKED):
        raise ValueError(f"weight_format must be 0, 1 or 2, got {weight_format}")
    w4 = weight_format == WEIGHTS_E2M1
    T, K = q.shape
    k = topk_ids.shape[1]
    E, twoI, Kw = w13.shape
    Kb = K // 2 if w4 else K
    if Kw != Kb or twoI % 2:
        raise ValueError(f"w13 must be [E, 2I, {Kb}], got {tuple(w13.shape)}")
    I = twoI // 2
    dev = q.device
    _need_like(q, (T, K), "q", torch.uint8, dev)
    _need_like(s, (T, _pairs(K), 2), "s", torch.uint8, dev)
    _need_like(topk_ids, (T, k), "topk_ids", torch.int32, dev)
    _need_like(topk_w, (T, k), "topk_w", torch.float32, dev)
    _need_like(w13, (E, twoI, Kb), "w13", torch.uint8, dev)
    _need_like(w13_s, (E, twoI, _pairs(K), 2), "w13_s", torch.uint8, dev)
    _need_like(w2, (E, K, I // 2 if w4 else I), "w2", torch.uint8, dev)
    _need_like(w2_s, (E, K, _pairs(I), 2), "w2_s", torch.uint8, dev)
    if out is not None:
        _need_like(out, (T, K), "out", torch.bfloat16, dev)
    if workspace is not None:
        _need_workspace(workspace, forward_workspace_size(T, K, I, E, k), dev)
    _need_gpu(q, "q")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return moe_mxfp8_forward_mx(q, s, topk_ids, topk_w, w13, w13_s, w2, w2_s, weight_format, out, workspace)
    if out is None:
        out = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = forward_workspace(T, K, I, E, k, dev)
    rc = load().moe_mxfp8_forward_mx(q.data_ptr(), s.data_ptr(), topk_ids.data_ptr(), topk_w.data_ptr(),
                                     weight_format, w13.data_ptr(), w13_s.data_ptr(), w2.data_ptr(), w2_s.data_ptr(),
                                     T, K, I, E, k, out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                     _raw_stream(dev.index))
    if rc:
        _check(rc, "moe_mxfp8_forward_mx")
    return out


ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def linear_fused_workspace_size(T, K, N, x_is_mx):
    return int(load().mx_linear_fused_workspace_size(T, K, N, int(x_is_mx)))


LINEAR_KERNELS = ("32x32", "64x64", "64x96", "64x64 twice per CU", "128x128", "256x128", "256x256", "32x32 bf16")


def linear_fused_kernel(T, K, N, x_is_mx):
    """Which of LINEAR_KERNELS (named by their tiles, weight rows x tokens)
    mx_linear_fused takes for a size on the current device."""
    index = load().mx_linear_fused_kernel(T, K, N, int(x_is_mx))
    if index < 0:
        _check(index, "mx_linear_fused_kernel")
    return LINEAR_KERNELS[index]


def mx_linear_fused(x, w, w_s, x_s=None, bias=None, act="none", residual=None, quantize_out=False, out=None,
                    workspace=None, stream=None):
    """Dense MXFP8 linear with its epilogue: act(x . w^T + bias) + residual, the
    epilogue in fp32 and rounded once.  The product is the scaled matrix
    instruction's: within 8 consecutive k each term is truncated to 13 bits
    below the largest one, off by less than 2^-10 of it together; these add in
    fp32.

    x: bf16 [T, K], or uint8 [T, K] with x_s uint8 [T, ceil(K/64), 2]; w, w_s:
    uint8 [N, K], [N, ceil(K/64), 2] (as mx_quantize makes them); bias: bf16 or
    fp32 [N]; act: a key of ACTIVATIONS; residual: bf16 [T, N].
    Returns y bf16 [T, N], or with ``quantize_out`` its MXFP8 (yq uint8 [T, N],
    ys uint8 [T, ceil(N/64), 2]).  ``out`` gives that tensor or pair instead
    (y may be the residual)."""
    mx_in = x_s is not None
    _need(x, _U8 if mx_in else _BF16, "x", 2)
    if type(w) is not _Tensor or w.dim() != 2:
        _need(w, _U8, "w", 2)
    T, K = x.shape
    N = w.shape[0]
    dev = x.device
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if mx_in:
        _need_like(x_s, (T, _pairs(K), 2), "x_s", _U8, dev)
    _need_like(w, (N, K), "w", _U8, dev)
    _need_like(w_s, (N, _pairs(K), 2), "w_s", _U8, dev)
    btype = TYPE_BF16
    if bias is not None:
        if isinstance(bias, _Tensor) and bias.dtype is _F32:
            btype = TYPE_F32
        _need_like(bias, (N,), "bias", _F32 if btype else _BF16, dev)
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    if residual is not None:
        _need_like(residual, (T, N), "residual", _BF16, dev)
    if out is not None:
        quantize_out = isinstance(out, (tuple, list))
    y = yq = ys = None
    if quantize_out:
        yq, ys = out if out is not None else (None, None)
        if out is not None:
            _need_like(yq, (T, N), "yq", _U8, dev)
            _need_like(ys, (T, _pairs(N), 2), "ys", _U8, dev)
    elif out is not None:
        y = out
        _need_like(y, (T, N), "out", _BF16, dev)
    lib = load()
    need = 0 if mx_in else lib.mx_linear_fused_workspace_size(T, K, N, 0)
    if workspace is not None:
        _need_workspace(workspace, need, dev)
    _need_gpu(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return mx_linear_fused(x, w, w_s, x_s, bias, act, residual, quantize_out, out, workspace)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=_U8, device=dev)
    if out is None:
        if quantize_out:
            yq = torch.empty((T, N), dtype=_U8, device=dev)
            ys = torch.empty((T, _pairs(N), 2), dtype=_U8, device=dev)
        else:
            y = torch.empty((T, N), dtype=_BF16, device=dev)
    rc = lib.mx_linear_fused(x.data_ptr(), _addr(x_s), w.data_ptr(), w_s.data_ptr(), _addr(bias), btype,
                             ACTIVATIONS[act], _addr(residual), T, K, N, _addr(y), _addr(yq), _addr(ys),
                             _addr(workspace), 0 if workspace is None else workspace.numel(),
                             _raw_stream(dev.index))
    if rc:
        _check(rc, "mx_linear_fused")
    return (yq, ys) if quantize_out else y


_I8, _I32 = torch.int8, torch.int32


def int8_quantize(x, out=None, stream=None):
    """bf16 rows [..., K] (rows may be strided) to int8 with one fp32 scale per
    row: s = max(amax / 127, 2^-126), q = round(x / s), in the fp32 steps that
    include/mxmoe.h gives; a row with a NaN or an infinity gets that scale and
    codes 0.  The tokens of int8_linear and gmm_int8, or their
    weights at load time ([N, K], [E, N, K]: a scale per output channel).
    Returns (q int8 [..., K], s fp32 [...]); ``out`` gives the two instead."""
    if type(x) is not _Tensor or x.dtype is not _BF16:
        _need(x, _BF16, "x")
    shape, dev = x.shape, x.device
    if x.is_cuda:   # before _rows, whose copy of strided leading dims belongs to the stream of the call
        there = _elsewhere(dev, stream)
        if there is not None:
            with there:
                return int8_quantize(x, out)
    if not shape or shape[-1] == 0:
        raise ValueError("x must have at least one element per row")
    x2, ldx = _rows(x, "x")
    if out is not None:
        q, s = out
        _need_like(q, shape, "q", _I8, dev)
        _need_like(s, shape[:-1], "s", _F32, dev)
    _need_gpu(x, "x")
    if out is None:
        q = torch.empty(shape, dtype=_I8, device=dev)
        s = torch.empty(shape[:-1], dtype=_F32, device=dev)
    rc = load().int8_quantize(x2.data_ptr(), x2.shape[0], shape[-1], ldx, q.data_ptr(), s.data_ptr(),
                              _raw_stream(dev.index))
    if rc:
        _check(rc, "int8_quantize")
    return q, s


def int8_linear_workspace_size(T, K, N, x_is_int8):
    return int(load().int8_linear_workspace_size(T, K, N, int(x_is_int8)))


INT8_KERNELS = ("32x16", "32x16 wide", "32x32", "48x48", "64x64", "128x128", "256x256", "32x16 bf16")


def int8_linear_kernel(T, K, N, x_is_int8):
    """Which of INT8_KERNELS (named by their tiles, weight rows x rows of x)
    int8_linear takes for a size on the current device."""
    index = load().int8_linear_kernel(T, K, N, int(x_is_int8))
    if index < 0:
        _check(index, "int8_linear_kernel")
    return INT8_KERNELS[index]


def gmm_int8_kernel(M, N, K, E, swiglu=False):
    """Which of INT8_KERNELS gmm_int8 takes for a size on the current device."""
    index = load().gmm_int8_kernel(M, N, K, E, int(swiglu))
    if index < 0:
        _check(index, "gmm_int8_kernel")
    return INT8_KERNELS[index]


def int8_linear(x, w, w_s, x_s=None, bias=None, act="none", residual=None, out=None, workspace=None, stream=None):
    """Dense INT8 linear with its epilogue: act((x . w^T) x_s w_s + bias) +
    residual, the product exact, the rest in fp32 and rounded once.

    x: bf16 [T, K], or int8 [T, K] with x_s fp32 [T]; w, w_s: int8 [N, K], fp32
    [N] (as int8_quantize makes them); bias: bf16 or fp32 [N]; act: a key of
    ACTIVATIONS; residual: bf16 [T, N].  Returns y bf16 [T, N]; ``out`` gives it
    instead (and may be the residual)."""
    int8_in = x_s is not None
    _need(x, _I8 if int8_in else _BF16, "x", 2)
    if type(w) is not _Tensor or w.dim() != 2:
        _need(w, _I8, "w", 2)
    T, K = x.shape
    N = w.shape[0]
    dev = x.device
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if int8_in:
        _need_like(x_s, (T,), "x_s", _F32, dev)
    _need_like(w, (N, K), "w", _I8, dev)
    _need_like(w_s, (N,), "w_s", _F32, dev)
    btype = TYPE_BF16
    if bias is not None:
        if isinstance(bias, _Tensor) and bias.dtype is _F32:
            btype = TYPE_F32
        _need_like(bias, (N,), "bias", _F32 if btype else _BF16, dev)
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    if residual is not None:
        _need_like(residual, (T, N), "residual", _BF16, dev)
    if out is not None:
        _need_like(out, (T, N), "out", _BF16, dev)
    lib = load()
    need = 0 if int8_in else lib.int8_linear_workspace_size(T, K, N, 0)
    if workspace is not None:
        _need_workspace(workspace, need, dev)
    _need_gpu(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return int8_linear(x, w, w_s, x_s, bias, act, residual, out, workspace)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=_U8, device=dev)
    if out is None:
        out = torch.empty((T, N), dtype=_BF16, device=dev)
    rc = lib.int8_linear(x.data_ptr(), _addr(x_s), w.data_ptr(), w_s.data_ptr(), _addr(bias), btype, ACTIVATIONS[act],
                         _addr(residual), T, K, N, out.data_ptr(), _addr(workspace),
                         0 if workspace is None else workspace.numel(), _raw_stream(dev.index))
    if rc:
        _check(rc, "int8_linear")
    return out


def gmm_int8(a, a_s, w, w_s, group_list, group_list_type=GROUP_COUNT, swiglu=False, out=None, stream=None):
    """Grouped INT8 product of rows sorted by expert: a int8 [M, K], a_s fp32 [M],
    w int8 [E, N, K], w_s fp32 [E, N], group_list int64 [E].  With ``swiglu`` w
    holds 2 N rows per expert, gate then up, and y = silu(gate) * up.  Returns y
    bf16 [M, N]; rows that no expert owns are not written."""
    _need(a, _I8, "a", 2)
    _need(w, _I8, "w", 3)
    M, K = a.shape
    E, rows = w.shape[:2]
    if swiglu and rows % 2:
        raise ValueError(f"w must be [E, 2N, {K}] with swiglu, got {tuple(w.shape)}")
    N = rows // 2 if swiglu else rows
    dev = a.device
    if not a.is_contiguous():
        raise ValueError("a must be contiguous")
    _need_like(a_s, (M,), "a_s", _F32, dev)
    _need_like(w, (E, rows, K), "w", _I8, dev)
    _need_like(w_s, (E, rows), "w_s", _F32, dev)
    _need_like(group_list, (E,), "group_list", torch.int64, dev)
    if out is not None:
        _need_like(out, (M, N), "out", _BF16, dev)
    _need_gpu(a, "a")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return gmm_int8(a, a_s, w, w_s, group_list, group_list_type, swiglu, out)
    if out is None:
        out = torch.empty((M, N), dtype=_BF16, device=dev)
    rc = load().gmm_int8(a.data_ptr(), a_s.data_ptr(), w.data_ptr(), w_s.data_ptr(), group_list.data_ptr(),
                         group_list_type, 1 if swiglu else 0, M, N, K, E, out.data_ptr(), _raw_stream(dev.index))
    if rc:
        _check(rc, "gmm_int8")
    return out


_ELEMENT_BYTES = {torch.bfloat16: 2, torch.float16: 2, torch.float32: 4, torch.int8: 1, torch.uint8: 1}   # (the usual ones)


def moe_permute(x, topk_ids, E, x_s=None, out=None, workspace=None, stream=None):
    """Token rows sorted by expert, as they are: x [T, K] of any type of 1, 2 or 4
    bytes (rows may be strided), topk_ids int32 [T, k]; x_s fp32 [T] (the scales
    of int8 rows) goes along.  Returns (xp [T*k, K], xp_s [T*k] or None,
    sorted_row, expanded_row_idx, group_list), the maps as moe_route_quant's;
    ``out`` gives the five instead.  Rows behind the last expert's (ids outside
    [0, E) are dropped) stay as they are.  The results carry no autograd graph: the
    gradient with respect to x is moe_unpermute of xp's gradient, without weights."""
    if not isinstance(x, _Tensor):
        _need(x, None, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must have 2 dims, got {len(shape)}")
    size = _ELEMENT_BYTES.get(x.dtype)
    if size is None:
        size = x.element_size()
        if size not in (1, 2, 4) or x.is_complex():
            raise TypeError(f"x must be of a type of 1, 2 or 4 bytes, got {x.dtype}")
    if type(topk_ids) is not _Tensor or topk_ids.dim() != 2:
        _need(topk_ids, _I32, "topk_ids", 2)
    T, K = shape
    if K == 0:
        raise ValueError("x must have at least one element per row")
    k = topk_ids.shape[1]
    M = T * k
    dev = x.device
    x2, ldx = (x, K) if x.is_contiguous() else _rows(x, "x")
    _need_like(topk_ids, (T, k), "topk_ids", _I32, dev)
    if x_s is not None:
        _need_like(x_s, (T,), "x_s", _F32, dev)
    if out is not None:
        xp, xps, sr, eri, gl = out
        _need_like(xp, (M, K), "xp", x.dtype, dev)
        if (xps is None) != (x_s is None):
            raise ValueError("xp_s goes with x_s")
        if xps is not None:
            _need_like(xps, (M,), "xp_s", _F32, dev)
        _need_like(sr, (M,), "sorted_row", _I32, dev)
        _need_like(eri, (M,), "expanded_row_idx", _I32, dev)
        _need_like(gl, (E,), "group_list", torch.int64, dev)
    lib = load()
    need = lib.moe_route_quant_workspace_size(T, k, E)
    if workspace is not None:
        _need_workspace(workspace, need, dev)
    _need_gpu(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return moe_permute(x, topk_ids, E, x_s, out, workspace)
    if out is None:
        xp = torch.empty((M, K), dtype=x.dtype, device=dev)
        xps = torch.empty(M, dtype=_F32, device=dev) if x_s is not None else None
        sr = torch.empty(M, dtype=_I32, device=dev)
        eri = torch.empty(M, dtype=_I32, device=dev)
        gl = torch.empty(E, dtype=torch.int64, device=dev)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=_U8, device=dev)
    rc = lib.moe_permute(x2.data_ptr(), ldx, size, _addr(x_s), topk_ids.data_ptr(), T, K, k, E, xp.data_ptr(),
                         _addr(xps), sr.data_ptr(), eri.data_ptr(), gl.data_ptr(), _addr(workspace),
                         0 if workspace is None else workspace.numel(), _raw_stream(dev.index))
    if rc:
        _check(rc, "moe_permute")
    return xp, xps, sr, eri, gl


TYPE_F16 = 2
_ROW_TYPES = {torch.bfloat16: TYPE_BF16, torch.float32: TYPE_F32, torch.float16: TYPE_F16}


def _row_type(t, name):
    """The rows' type by number."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    kind = _ROW_TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have 2 dims, got {len(shape)}")
    if shape[1] == 0:
        raise ValueError(f"{name} must have at least one element per row")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return kind


def _tokens(expanded_row_idx, k, dev):
    """T of expanded_row_idx [T*k] (of any shape)."""
    if not isinstance(k, int) or k <= 0:
        raise ValueError(f"k must be a positive int, got {k!r}")
    e = expanded_row_idx
    if not (type(e) is _Tensor and e.dtype is _I32 and e.is_contiguous() and e.device == dev):
        _need(e, _I32, "expanded_row_idx")
        _need_shape(e, e.shape, "expanded_row_idx", _I32, dev)
    n = e.numel()
    if n % k:
        raise ValueError(f"expanded_row_idx must hold T*k entries, got {n} with k = {k}")
    return n // k


def moe_unpermute(y, expanded_row_idx, k, topk_w=None, out=None, stream=None):
    """Expert rows back to their tokens: out[t] = sum_j topk_w[t, j] *
    y[expanded_row_idx[t*k+j]], in fp32 and rounded once; without weights their
    plain sum (the gradient of moe_permute).  y: bf16, fp16 or fp32 [M, K] of any
    K; topk_w: fp32 [T, k].  Entries outside [0, M) are skipped.  Returns out
    [T, K] of y's type, which carries no autograd graph: moe_unpermute_backward
    gives the gradients."""
    kind = _row_type(y, "y")
    M, K = y.shape
    dev = y.device
    T = _tokens(expanded_row_idx, k, dev)
    if topk_w is not None:
        _need_like(topk_w, (T, k), "topk_w", _F32, dev)
    if out is not None:
        _need_like(out, (T, K), "out", y.dtype, dev)
    _need_gpu(y, "y")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return moe_unpermute(y, expanded_row_idx, k, topk_w, out)
    if out is None:
        out = torch.empty((T, K), dtype=y.dtype, device=dev)
    rc = load().moe_unpermute(y.data_ptr(), kind, _addr(topk_w), expanded_row_idx.data_ptr(), T, K, k, M,
                              out.data_ptr(), _raw_stream(dev.index))
    if rc:
        _check(rc, "moe_unpermute")
    return out


def moe_unpermute_backward(dout, expanded_row_idx, k, topk_w=None, y=None, out=None, stream=None):
    """The gradients of moe_unpermute (and moe_finalize): dy[p] = topk_w[t, j] *
    dout[t] for p = expanded_row_idx[t*k+j], and with ``y`` also dw[t, j] =
    <dout[t], y[p]> in fp32 (0 for a dropped entry).  dout [T, K] and y [M, K]:
    bf16, fp16 or fp32; M = T*k without y.  Returns (dy [M, K], dw [T, k] or
    None); ``out`` gives the two instead.  Rows that no entry names are zeros in a
    dy made here, which is cleared first (a pass over dy more: 16384 tokens of 2048
    bf16 with 8 rows each 330 us, 224 with ``out``), and stay as they are in one
    given: where entries may be dropped, clear those rows."""
    kind = _row_type(dout, "dout")
    rows, K = dout.shape
    dev = dout.device
    T = _tokens(expanded_row_idx, k, dev)
    if rows != T:
        raise ValueError(f"dout must have {T} rows, got {rows}")
    if topk_w is not None:
        _need_like(topk_w, (T, k), "topk_w", _F32, dev)
    M = T * k
    dtype = dout.dtype
    if y is not None:
        if type(y) is not _Tensor or y.dim() != 2:
            _need(y, dtype, "y", 2)
        M = y.shape[0]
        _need_like(y, (M, K), "y", dtype, dev)
    if out is not None:
        dy, dw = out
        if y is None:
            _need(dy, dtype, "dy", 2)
            M = dy.shape[0]
        _need_like(dy, (M, K), "dy", dtype, dev)
        if (dw is None) != (y is None):
            raise ValueError("dw goes with y")
        if dw is not None:
            _need_like(dw, (T, k), "dw", _F32, dev)
    _need_gpu(dout, "dout")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return moe_unpermute_backward(dout, expanded_row_idx, k, topk_w, y, out)
    if out is None:
        dy = torch.zeros((M, K), dtype=dtype, device=dev)
        dw = torch.empty((T, k), dtype=_F32, device=dev) if y is not None else None
    rc = load().moe_unpermute_backward(dout.data_ptr(), kind, _addr(y), _addr(topk_w), expanded_row_idx.data_ptr(), T,
                                       K, k, M, dy.data_ptr(), _addr(dw), _raw_stream(dev.index))
    if rc:
        _check(rc, "moe_unpermute_backward")
    return dy, dw
