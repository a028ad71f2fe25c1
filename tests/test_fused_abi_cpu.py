"""Host checks of the operators around the expert layer that need no GPU: the
C entry points' statuses (nothing is enqueued) and the binding's argument
checks on CPU tensors (shape errors come before the GPU-residency check)."""

import ctypes
import math
import os

import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
BIG = [1 << 31, 1 << 40, (1 << 63) - 1]
NEG = [-1, -(1 << 63)]


def at(i):
    """A distinct, 256-byte aligned address, 1 TiB apart (never dereferenced)."""
    return ctypes.c_void_p((i + 1) << 40)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.lib_path()):
        pytest.fail("libmxmoe.so is not built (run python -m mxfp8_block_scaled_topk_amd.build)")
    return mx.load()


def norm(lib, x=at(0), ldx=64, res=at(1), ldr=64, w=at(2), wt=0, eps=1e-6, rows=4, kd=64, ro=at(3), y=at(4), q=at(5),
         s=at(6)):
    return lib.mx_add_rmsnorm(x, ldx, res, ldr, w, wt, eps, rows, kd, ro, y, q, s, None)


def test_norm_validation(lib):
    for kw in (dict(rows=-1), dict(kd=0), dict(ldx=63), dict(ldr=10), dict(wt=2), dict(wt=-1), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(eps=1e-40), dict(q=None), dict(s=None),
               dict(res=None), dict(x=None), dict(w=None), dict(y=None, q=None, s=None)):
        assert norm(lib, **kw) == INVALID, kw
    for v in NEG:
        assert norm(lib, rows=v) == INVALID and norm(lib, kd=v) == INVALID
    for v in BIG:
        assert norm(lib, rows=v) == UNSUPPORTED
        assert norm(lib, ldx=v) == UNSUPPORTED and norm(lib, ldr=v) == UNSUPPORTED
    assert norm(lib, kd=(1 << 24) + 1, ldx=1 << 25, ldr=1 << 25) == UNSUPPORTED
    assert norm(lib, x=ctypes.c_void_p(0x1001)) == UNSUPPORTED          # odd address of bf16
    assert norm(lib, w=ctypes.c_void_p(0x1002), wt=1) == UNSUPPORTED    # fp32 weight on 2 bytes
    assert norm(lib, rows=0, x=None, w=None, y=None, ro=None, res=None) == OK


def test_norm_overlap(lib):
    a = ctypes.c_void_p
    base = 1 << 40
    assert norm(lib, q=a(base), s=a(base + 10)) == INVALID                 # q over x (and s inside it)
    assert norm(lib, ro=a(base + 2)) == INVALID                            # residual_out into x, shifted
    assert norm(lib, ro=at(0), ldx=72) == INVALID                          # over x whose rows are further apart
    assert norm(lib, ro=at(4)) == INVALID                                  # two outputs
    assert norm(lib, y=at(2)) == INVALID                                   # over the weight
    assert "overlap" in mx.last_error()


def lin(lib, x=at(0), xs=at(1), w=at(2), ws=at(3), b=at(4), bt=0, act=0, r=at(5), T=4, K=64, N=96, y=at(6), yq=None,
        ys=None, wsp=None, wsb=0):
    return lib.mx_linear_fused(x, xs, w, ws, b, bt, act, r, T, K, N, y, yq, ys, wsp, wsb, None)


def test_linear_fused_validation(lib):
    for kw in (dict(T=-1), dict(K=0), dict(N=0), dict(bt=2), dict(act=-1), dict(act=5), dict(yq=at(7)),
               dict(y=None, yq=at(7)), dict(yq=at(7), ys=at(8)), dict(x=None), dict(w=None), dict(ws=None),
               dict(y=None)):
        assert lin(lib, **kw) == INVALID, kw
    for v in NEG:
        assert lin(lib, T=v) == INVALID and lin(lib, K=v) == INVALID and lin(lib, N=v) == INVALID
    for v in BIG:
        assert lin(lib, T=v) == UNSUPPORTED and lin(lib, N=v) == UNSUPPORTED
        assert lin(lib, K=v // 32 * 32) == UNSUPPORTED
    assert lin(lib, K=65) == UNSUPPORTED and "multiple of 32" in mx.last_error()
    assert lin(lib, K=(1 << 20) + 32) == UNSUPPORTED
    a = ctypes.c_void_p
    assert lin(lib, x=a(0x1008)) == UNSUPPORTED and lin(lib, w=a(0x1008)) == UNSUPPORTED
    assert lin(lib, xs=a(0x1002)) == UNSUPPORTED and lin(lib, ws=a(0x1002)) == UNSUPPORTED
    assert lin(lib, b=a(0x1002), bt=1) == UNSUPPORTED and lin(lib, y=a(0x1001)) == UNSUPPORTED
    # bf16 tokens past what workgroups quantise for themselves need a workspace
    need = mx.linear_fused_workspace_size(64, 64, 96, False)
    assert need >= 64 * 64 + 64 * 2
    assert lin(lib, xs=None, T=64) == INVALID and lin(lib, xs=None, T=64, wsp=at(9), wsb=need - 1) == WORKSPACE
    assert lin(lib, xs=None, T=64, wsp=a(0x1010), wsb=need) == UNSUPPORTED
    assert lin(lib, T=0, x=None, xs=None, w=None, ws=None, y=None) == OK
    assert mx.linear_fused_workspace_size(64, 64, 96, True) == 0
    assert mx.linear_fused_workspace_size(64, 65, 96, False) == 0
    for v in NEG + BIG:
        assert mx.linear_fused_workspace_size(v, 64, 96, False) == 0
        assert mx.linear_fused_workspace_size(64, 64, v, False) == 0


def test_linear_fused_overlap(lib):
    a = ctypes.c_void_p
    assert lin(lib, y=at(2)) == INVALID                                    # y over w
    assert lin(lib, y=a((6 << 40) + 2)) == INVALID                         # y into the residual, shifted
    assert lin(lib, y=None, r=None, yq=at(0), ys=at(8)) == INVALID         # yq over x
    assert lin(lib, y=None, r=None, yq=at(7), ys=a((8 << 40) + 16)) == INVALID   # ys inside yq
    # the workspace, where bf16 tokens are quantised to, over them or over the weights
    for other in (dict(x=at(7)), dict(w=at(7)), dict(b=at(7)), dict(r=at(7)), dict(y=at(7))):
        assert lin(lib, T=64, xs=None, wsp=at(7), wsb=1 << 20, **other) == INVALID, other
    assert "overlap" in mx.last_error()


def test_route_mx_and_forward_mx_validation(lib):
    def route(T, K, k, E, ws=1 << 30, q=at(0), s=at(1), wsp=at(9)):
        return lib.moe_route_mx(q, s, at(2), T, K, k, E, at(3), at(4), at(5), at(6), at(7), wsp, ws, None)
    assert route(64, 256, 9, 8) == INVALID and "moe_route_mx" in mx.last_error()
    assert route(64, 256, 0, 8) == INVALID and route(64, 100, 2, 8) == UNSUPPORTED
    assert route(64, 256, 2, 2048) == UNSUPPORTED and route(300, 256, 2, 8, ws=0) == WORKSPACE
    assert route(64, 256, 2, 8, s=None) == INVALID
    assert route(64, 256, 2, 8, q=ctypes.c_void_p(0x1008)) == UNSUPPORTED
    assert route(300, 256, 2, 8, wsp=ctypes.c_void_p(0x1004)) == UNSUPPORTED

    bufs = [at(i) for i in range(8)] + [at(9)]   # q s ids xq xs sorted_row expanded_row_idx group_list workspace
    for i in range(9):
        for o in range(max(i + 1, 3), 9):
            b = list(bufs)
            b[o] = b[i]
            rc = lib.moe_route_mx(*b[:3], 300, 256, 2, 8, *b[3:], 1 << 30, None)
            assert rc == INVALID and "overlap" in mx.last_error(), (i, o)

    def fwd(fmt, T, K, I, E, k, ws=1 << 40, s=at(1)):
        return lib.moe_mxfp8_forward_mx(at(0), s, at(2), at(3), fmt, at(4), at(5), at(6), at(7), T, K, I, E, k, at(8),
                                        at(9), ws, None)
    for fmt in (0, 1, 2):
        assert fwd(fmt, 64, 256, 96, 8, 2) == UNSUPPORTED and fwd(fmt, 64, 256, 128, 8, 9) == INVALID
        assert fwd(fmt, 64, 256, 128, 8, 2, ws=16) == WORKSPACE and fwd(fmt, 64, 256, 128, 8, 2, s=None) == INVALID
    assert fwd(3, 64, 256, 128, 8, 2) == INVALID and fwd(-1, 64, 256, 128, 8, 2) == INVALID


def _raises(fn, pattern):
    with pytest.raises((ValueError, TypeError), match=pattern):
        fn()


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_binding_norm_checks(lib):
    x, w = _bf(4, 100), _bf(100)
    _raises(lambda: mx.mx_add_rmsnorm(x, w), "on the GPU")
    _raises(lambda: mx.mx_add_rmsnorm(x.float(), w), "x must be torch.bfloat16")
    _raises(lambda: mx.mx_add_rmsnorm(x, w.double()), "weight must be torch.bfloat16")
    _raises(lambda: mx.mx_add_rmsnorm(x, _bf(99)), "weight must have shape")
    _raises(lambda: mx.mx_add_rmsnorm(x, None), "weight must be a torch.Tensor")
    _raises(lambda: mx.mx_add_rmsnorm(None, w), "x must be a torch.Tensor")
    _raises(lambda: mx.mx_add_rmsnorm(x, w, x.float()), "residual must be torch.bfloat16")
    _raises(lambda: mx.mx_add_rmsnorm(torch.nn.Parameter(x), torch.nn.Parameter(w)), "on the GPU")   # as tensors
    _raises(lambda: mx.mx_add_rmsnorm(x, w, _bf(4, 99)), "residual must have shape")
    _raises(lambda: mx.mx_add_rmsnorm(_bf(100, 4).t(), w), "unit stride")
    _raises(lambda: mx.mx_add_rmsnorm(_bf(1, 100).expand(4, 100), w), "repeat its rows")
    _raises(lambda: mx.mx_add_rmsnorm(_bf(4, 0), _bf(0)), "at least one element")
    _raises(lambda: mx.mx_add_rmsnorm(x, w, out=(_u8(4, 100), _u8(4, 1, 2), None, None)), "s must have shape")
    _raises(lambda: mx.mx_add_rmsnorm(x, w, out=(None, None, None, _bf(100, 4).t())), "y must be contiguous")
    _raises(lambda: mx.mx_add_rmsnorm(x, w, x, out=(None, None, _bf(4, 50), None)), "residual_out must have shape")


def test_binding_linear_fused_checks(lib):
    x, w, ws = _bf(10, 96), _u8(33, 96), _u8(33, 2, 2)
    _raises(lambda: mx.mx_linear_fused(x, w, ws), "on the GPU")
    _raises(lambda: mx.mx_linear_fused(x, w, ws, x_s=_u8(10, 2, 2)), "x must be torch.uint8")
    _raises(lambda: mx.mx_linear_fused(_u8(10, 96), w, ws), "x must be torch.bfloat16")
    _raises(lambda: mx.mx_linear_fused(_u8(10, 96), w, ws, x_s=_u8(10, 1, 2)), "x_s must have shape")
    _raises(lambda: mx.mx_linear_fused(x, _u8(33, 64), ws), "w must have shape")
    _raises(lambda: mx.mx_linear_fused(x, w, _u8(33, 1, 2)), "w_s must have shape")
    _raises(lambda: mx.mx_linear_fused(x, w, ws, bias=torch.zeros(32)), "bias must have shape")
    _raises(lambda: mx.mx_linear_fused(x, w, ws, bias=torch.zeros(33, dtype=torch.float64)), "bias must be")
    _raises(lambda: mx.mx_linear_fused(x, w, ws, act="tanh"), "act must be one of")
    _raises(lambda: mx.mx_linear_fused(x, w, ws, residual=_bf(10, 32)), "residual must have shape")
    _raises(lambda: mx.mx_linear_fused(x, w, ws, out=_bf(10, 32)), "out must have shape")
    _raises(lambda: mx.mx_linear_fused(x, w, ws, out=(_u8(10, 33), _u8(10, 2, 2))), "ys must have shape")
    _raises(lambda: mx.mx_linear_fused(_bf(96, 10).t(), w, ws), "x must be contiguous")
    _raises(lambda: mx.mx_linear_fused(x, w[0], ws), "w must have 2 dims")
    _raises(lambda: mx.mx_linear_fused(x, None, ws), "w must be a torch.Tensor")
    _raises(lambda: mx.mx_linear_fused(x, w.int(), ws), "w must be torch.uint8")
    _raises(lambda: mx.mx_linear_fused(x, torch.nn.Parameter(w, requires_grad=False), ws), "on the GPU")   # as a tensor
    _raises(lambda: mx.mx_linear_fused(_bf(100, 96), w, ws, workspace=_u8(16)), "workspace has 16 bytes")


def test_binding_route_mx_and_forward_mx_checks(lib):
    q, s, ids = _u8(8, 256), _u8(8, 4, 2), torch.zeros(8, 2, dtype=torch.int32)
    _raises(lambda: mx.moe_route_mx(q, s, ids, 4), "on the GPU")
    _raises(lambda: mx.moe_route_mx(q, _u8(8, 3, 2), ids, 4), "s must have shape")
    _raises(lambda: mx.moe_route_mx(q, s, ids[:7], 4), "topk_ids must have shape")
    _raises(lambda: mx.moe_route_mx(q, s, ids.long(), 4), "topk_ids must be torch.int32")
    _raises(lambda: mx.moe_route_mx(q, s, ids[0], 4), "topk_ids must have 2 dims")
    _raises(lambda: mx.moe_route_mx(q, s, None, 4), "topk_ids must be a torch.Tensor")
    _raises(lambda: mx.moe_route_mx(_u8(256, 8).t(), s, ids, 4), "q must be contiguous")
    E, I = 4, 128
    args = (q, s, ids, torch.zeros(8, 2), _u8(E, 2 * I, 256), _u8(E, 2 * I, 4, 2), _u8(E, 256, I), _u8(E, 256, 2, 2))
    _raises(lambda: mx.moe_mxfp8_forward_mx(*args), "on the GPU")
    _raises(lambda: mx.moe_mxfp8_forward_mx(*args, weight_format=3), "weight_format")
    _raises(lambda: mx.moe_mxfp8_forward_mx(*args, weight_format=mx.WEIGHTS_E2M1), "w13 must be")
    _raises(lambda: mx.moe_mxfp8_forward_mx(*args, out=_bf(8, 128)), "out must have shape")
    _raises(lambda: mx.moe_mxfp8_forward_mx(*args, workspace=_u8(64)), "workspace has 64 bytes")
