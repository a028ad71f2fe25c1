"""Host checks of the INT8 products and of the expert sort and its way back that
need no GPU: the C entry points' statuses (nothing is enqueued) and the binding's
argument checks on CPU tensors (shape errors come before the GPU-residency
check)."""

import ctypes
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


def odd(i, by):
    return ctypes.c_void_p(((i + 1) << 40) + by)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.lib_path()):
        pytest.fail("libmxmoe.so is not built (run python -m mxfp8_block_scaled_topk_amd.build)")
    return mx.load()


def quant(lib, x=at(0), rows=4, kd=64, ld=64, q=at(1), s=at(2)):
    return lib.int8_quantize(x, rows, kd, ld, q, s, None)


def test_quantize_validation(lib):
    for kw in (dict(rows=-1), dict(kd=0), dict(ld=63), dict(x=None), dict(q=None), dict(s=None), dict(q=at(0)),
               dict(s=odd(0, 64)), dict(s=odd(1, 128)), dict(q=odd(0, 511))):
        assert quant(lib, **kw) == INVALID, kw
    for v in NEG:
        assert quant(lib, rows=v) == INVALID and quant(lib, kd=v) == INVALID and quant(lib, ld=v) == INVALID
    for v in BIG:
        assert quant(lib, rows=v) == UNSUPPORTED and quant(lib, ld=v) == UNSUPPORTED
        assert quant(lib, kd=v, ld=v) == UNSUPPORTED
    assert quant(lib, kd=(1 << 24) + 1, ld=1 << 25) == UNSUPPORTED
    assert quant(lib, x=odd(0, 1)) == UNSUPPORTED and quant(lib, s=odd(2, 2)) == UNSUPPORTED
    assert quant(lib, rows=0, x=None, q=None, s=None) == OK


def lin(lib, T=4, K=64, N=96, x=at(0), xs=at(1), w=at(2), ws=at(3), b=at(4), bt=0, act=0, r=at(5), y=at(6), wsp=None, wsb=0):
    return lib.int8_linear(x, xs, w, ws, b, bt, act, r, T, K, N, y, wsp, wsb, None)


def test_linear_validation(lib):
    for kw in (dict(T=-1), dict(K=0), dict(N=0), dict(bt=2), dict(bt=-1), dict(act=5), dict(act=-1), dict(x=None),
               dict(w=None), dict(ws=None), dict(y=None), dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3)),
               dict(y=at(4)), dict(y=odd(5, 2)), dict(T=40, xs=None, wsp=None, wsb=1 << 20),
               dict(T=40, xs=None, wsp=at(0), wsb=1 << 20), dict(T=40, xs=None, wsp=at(6), wsb=1 << 20),
               dict(T=40, xs=None, wsp=at(5), wsb=1 << 20)):
        assert lin(lib, **kw) == INVALID, kw
    for v in NEG:
        for n in ("T", "K", "N"):
            assert lin(lib, **{n: v}) == INVALID, (n, v)
    for v in BIG:
        for n in ("T", "N"):
            assert lin(lib, **{n: v}) == UNSUPPORTED, (n, v)
    for kw in (dict(K=8), dict(K=72), dict(K=1 << 17), dict(K=1 << 20), dict(N=1 << 30), dict(N=1 << 27), dict(T=1 << 30, N=1 << 10),
               dict(x=odd(0, 8)), dict(w=odd(2, 8)), dict(xs=odd(1, 2)), dict(ws=odd(3, 1)), dict(b=odd(4, 1)),
               dict(b=odd(4, 2), bt=1), dict(r=odd(5, 1)), dict(y=odd(6, 1)), dict(xs=None, x=odd(0, 1), wsp=at(9), wsb=1 << 20),
               dict(T=40, xs=None, wsp=odd(9, 128), wsb=1 << 20)):
        assert lin(lib, **kw) == UNSUPPORTED, kw
    need = lib.int8_linear_workspace_size(40, 64, 96, 0)
    assert need >= 40 * 64 + 160 and lib.int8_linear_workspace_size(40, 64, 96, 1) == 0
    assert lib.int8_linear_workspace_size(4, 64, 96, 0) == 0   # few tokens are quantised in place
    assert lin(lib, T=40, xs=None, wsp=at(9), wsb=need - 1) == WORKSPACE
    for v in NEG + BIG + [0]:
        assert lib.int8_linear_workspace_size(40, v, 96, 0) == 0
    assert lin(lib, T=0, x=None, w=None, ws=None, y=None, b=None, r=None) == OK


def experts(lib, a=at(0), a_s=at(1), w=at(2), ws=at(3), gl=at(4), kind=1, swiglu=0, M=5, N=96, K=64, E=3, y=at(5)):
    return lib.gmm_int8(a, a_s, w, ws, gl, kind, swiglu, M, N, K, E, y, None)


def test_experts_validation(lib):
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(E=0), dict(E=-1), dict(kind=2), dict(kind=-1), dict(a=None),
               dict(a_s=None), dict(w=None), dict(ws=None), dict(gl=None), dict(y=None), dict(y=at(0)), dict(y=at(1)),
               dict(y=at(2)), dict(y=at(3)), dict(y=at(4)), dict(y=odd(2, 3 * 96 * 64 * 2 - 2), swiglu=1)):
        assert experts(lib, **kw) == INVALID, kw
    for v in NEG:
        for n in ("M", "N", "K", "E"):
            assert experts(lib, **{n: v}) == INVALID, (n, v)
    for v in BIG:
        for n in ("M", "N", "E"):
            assert experts(lib, **{n: v}) == UNSUPPORTED, (n, v)
    for kw in (dict(K=24), dict(K=1 << 17), dict(N=1 << 30), dict(N=1 << 27), dict(E=1025), dict(a=odd(0, 4)), dict(w=odd(2, 4)),
               dict(a_s=odd(1, 2)), dict(ws=odd(3, 2)), dict(gl=odd(4, 4)), dict(y=odd(5, 1)), dict(M=1 << 28, N=1 << 14)):
        assert experts(lib, **kw) == UNSUPPORTED, kw
    assert experts(lib, M=0, a=None, a_s=None, w=None, ws=None, y=None) == OK
    assert experts(lib, M=0, gl=None) == INVALID


def permute(lib, x=at(0), ldx=64, eb=2, xs=None, ids=at(1), T=4, K=64, k=2, E=8, xp=at(2), xps=None, sr=at(3), eri=at(4),
            gl=at(5), ws=None, wsb=0):
    return lib.moe_permute(x, ldx, eb, xs, ids, T, K, k, E, xp, xps, sr, eri, gl, ws, wsb, None)


def test_permute_validation(lib):
    for kw in (dict(T=-1), dict(K=0), dict(k=0), dict(E=0), dict(k=9), dict(eb=0), dict(eb=3), dict(eb=8), dict(ldx=63),
               dict(x=None), dict(ids=None), dict(xp=None), dict(sr=None), dict(eri=None), dict(gl=None), dict(xs=at(6)),
               dict(xps=at(6)), dict(T=200), dict(xp=at(0)), dict(sr=at(1)), dict(eri=at(3)), dict(gl=at(2)),
               dict(xs=at(6), xps=at(6)), dict(xs=at(6), xps=at(2))):
        assert permute(lib, **kw) == INVALID, kw
    for v in NEG:
        for n in ("T", "K", "k", "E", "ldx"):
            assert permute(lib, **{n: v}) == INVALID, (n, v)
    for v in BIG:
        assert permute(lib, T=v) == UNSUPPORTED and permute(lib, K=v, ldx=v) == UNSUPPORTED
        assert permute(lib, ldx=v) == UNSUPPORTED and permute(lib, E=v) == UNSUPPORTED
    for kw in (dict(K=(1 << 24) + 1, ldx=1 << 25), dict(k=257, E=1000), dict(E=1025), dict(T=1 << 27), dict(x=odd(0, 1)),
               dict(xp=odd(2, 1)), dict(xs=odd(6, 2), xps=at(7)), dict(xs=at(6), xps=odd(7, 1)), dict(ids=odd(1, 2)),
               dict(gl=odd(5, 4)), dict(T=200, ws=odd(9, 4), wsb=1 << 20), dict(eb=4, x=odd(0, 2))):
        assert permute(lib, **kw) == UNSUPPORTED, kw
    need = lib.moe_route_quant_workspace_size(200, 2, 8)
    assert need > 0 and permute(lib, T=200, ws=at(9), wsb=need - 1) == WORKSPACE
    assert permute(lib, T=200, ws=at(2), wsb=need) == INVALID


def back(lib, y=at(0), type=0, w=at(1), eri=at(2), T=4, K=64, k=2, M=8, out=at(3)):
    return lib.moe_unpermute(y, type, w, eri, T, K, k, M, out, None)


def grad(lib, d=at(0), type=0, y=at(1), w=at(2), eri=at(3), T=4, K=64, k=2, M=8, dy=at(4), dw=at(5)):
    return lib.moe_unpermute_backward(d, type, y, w, eri, T, K, k, M, dy, dw, None)


@pytest.mark.parametrize("call", [back, grad])
def test_unpermute_sizes(lib, call):
    for kw in (dict(T=-1), dict(K=0), dict(k=0), dict(M=-1), dict(type=3), dict(type=-1), dict(eri=None)):
        assert call(lib, **kw) == INVALID, kw
    for v in NEG:
        for n in ("T", "K", "k", "M"):
            assert call(lib, **{n: v}) == INVALID, (n, v)
    for v in BIG:
        for n in ("T", "K", "k", "M"):
            assert call(lib, **{n: v}) == UNSUPPORTED, (n, v)
    for kw in (dict(K=(1 << 24) + 1), dict(T=1 << 16, k=1 << 15), dict(w=odd(9, 2)), dict(eri=odd(9, 1)), dict(y=odd(9, 1)),
               dict(y=odd(9, 2), type=1), dict(y=odd(9, 1), type=2)):
        assert call(lib, **kw) == UNSUPPORTED, kw


def test_unpermute_validation(lib):
    for kw in (dict(y=None), dict(out=None), dict(out=at(0)), dict(out=at(1)), dict(out=odd(2, 28))):
        assert back(lib, **kw) == INVALID, kw
    assert back(lib, out=odd(3, 1)) == UNSUPPORTED
    assert back(lib, T=0, y=None, out=None, eri=None) == OK
    for kw in (dict(d=None), dict(dy=None), dict(y=None), dict(dy=at(0)), dict(dy=at(1)), dict(dy=at(2)), dict(dy=at(3)),
               dict(dw=at(0)), dict(dw=at(1)), dict(dw=at(2)), dict(dw=odd(4, 128))):
        assert grad(lib, **kw) == INVALID, kw
    assert grad(lib, dy=odd(4, 1)) == UNSUPPORTED and grad(lib, dw=odd(5, 2)) == UNSUPPORTED
    assert grad(lib, T=0, d=None, dy=None, y=None, dw=None, eri=None) == OK


def test_binding_checks():
    """On CPU tensors: what is wrong with the arguments comes before where they are."""
    bf, i8, f32, i32, i64 = torch.bfloat16, torch.int8, torch.float32, torch.int32, torch.int64
    z = torch.zeros
    good_x, good_ids = z(4, 64, dtype=bf), z(4, 2, dtype=i32)
    with pytest.raises(TypeError):
        mx.int8_quantize(z(4, 64))
    with pytest.raises(ValueError, match="unit stride"):
        mx.int8_quantize(z(64, 4, dtype=bf).t())
    with pytest.raises(ValueError, match="repeat"):
        mx.int8_quantize(z(1, 64, dtype=bf).expand(4, 64))
    with pytest.raises(ValueError, match="shape"):
        mx.int8_quantize(good_x, out=(z(4, 64, dtype=i8), z(5)))
    with pytest.raises(TypeError):
        mx.int8_quantize(good_x, out=(z(4, 64, dtype=torch.uint8), z(4)))
    with pytest.raises(ValueError, match="one element"):
        mx.int8_quantize(z(4, 0, dtype=bf))
    with pytest.raises(ValueError, match="on the GPU"):
        mx.int8_quantize(good_x)

    w, ws, xq, xs = z(96, 64, dtype=i8), z(96), z(4, 64, dtype=i8), z(4)
    for args, kw in (((good_x, w, ws), dict(x_s=xs)), ((xq, w, ws), {}), ((xq, w.float(), ws), dict(x_s=xs)),
                     ((xq, w, ws.double()), dict(x_s=xs)), ((xq, w, ws), dict(x_s=xs.to(bf)))):
        with pytest.raises(TypeError):
            mx.int8_linear(*args, **kw)
    for args, kw in (((xq, w[:, :32], ws), {}), ((xq, w, ws[:5]), {}), ((xq.t().contiguous().t(), w, ws), {}),
                     ((xq, w, ws), dict(bias=z(95))), ((xq, w, ws), dict(act="tanh")), ((xq, w, ws), dict(residual=z(4, 95, dtype=bf))),
                     ((xq, w, ws), dict(out=z(5, 96, dtype=bf)))):
        with pytest.raises(ValueError):
            mx.int8_linear(*args, x_s=xs, **kw)
    with pytest.raises(ValueError, match="on the GPU"):
        mx.int8_linear(xq, w, ws, x_s=xs)

    ew, ews, gl = z(3, 96, 64, dtype=i8), z(3, 96), z(3, dtype=i64)
    for a in ((good_x, xs, ew, ews, gl), (xq, xs, ew, ews, gl.int()), (xq, xs.double(), ew, ews, gl)):
        with pytest.raises(TypeError):
            mx.gmm_int8(*a)
    for a, kw in (((xq, xs, ew, ews, gl[:2]), {}), ((xq, z(5), ew, ews, gl), {}), ((xq, xs, ew[:, :, :48], ews, gl), {}),
                  ((xq, xs, ew[:, :95].contiguous(), ews[:, :95].contiguous(), gl), dict(swiglu=True)),
                  ((xq, xs, ew, ews, gl), dict(swiglu=True, out=z(4, 96, dtype=bf))), ((xq, xs, w, ews, gl), {})):
        with pytest.raises(ValueError):
            mx.gmm_int8(*a, **kw)
    with pytest.raises(ValueError, match="on the GPU"):
        mx.gmm_int8(xq, xs, ew, ews, gl)

    with pytest.raises(TypeError, match="1, 2 or 4"):
        mx.moe_permute(z(4, 64, dtype=torch.float64), good_ids, 8)
    with pytest.raises(TypeError):
        mx.moe_permute(good_x, good_ids.long(), 8)
    with pytest.raises(TypeError):
        mx.moe_permute([1.0], good_ids, 8)
    for kw in (dict(x_s=z(5)), dict(out=(z(8, 64, dtype=bf), z(8), z(8, dtype=i32), z(8, dtype=i32), z(8, dtype=i64))),
               dict(out=(z(8, 63, dtype=bf), None, z(8, dtype=i32), z(8, dtype=i32), z(8, dtype=i64)))):
        with pytest.raises(ValueError):
            mx.moe_permute(good_x, good_ids, 8, **kw)
    for x, ids in ((z(4, 0, dtype=bf), good_ids), (z(64, 4, dtype=bf).t(), good_ids), (good_x, z(5, 2, dtype=i32))):
        with pytest.raises(ValueError):
            mx.moe_permute(x, ids, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        mx.moe_permute(good_x, good_ids, 8)

    y, eri = z(8, 64, dtype=torch.float16), z(8, dtype=i32)
    with pytest.raises(TypeError):
        mx.moe_unpermute(y.double(), eri, 2)
    with pytest.raises(TypeError):
        mx.moe_unpermute(y, eri.long(), 2)
    for a, kw in (((y, eri, 3), {}), ((y, eri, 0), {}), ((y, eri, 2.0), {}), ((y.t(), eri, 2), {}), ((y, eri, 2), dict(topk_w=z(4, 3))),
                  ((y, eri, 2), dict(out=z(4, 63, dtype=torch.float16))), ((y[:, :0], eri, 2), {}), ((y, eri, 2), {})):
        with pytest.raises(ValueError):
            mx.moe_unpermute(*a, **kw)
    d = z(4, 64, dtype=torch.float16)
    for kw in (dict(y=y.float()), dict(out=(y.float(), None))):
        with pytest.raises(TypeError):
            mx.moe_unpermute_backward(d, eri, 2, **kw)
    for a, kw in (((d[:3], eri, 2), {}), ((d, eri, 2), dict(out=(y, z(4, 2)))), ((d, eri, 2), dict(y=y, out=(y, None))),
                  ((d, eri, 2), dict(y=y[:, :32].contiguous())), ((d, eri, 2), {})):
        with pytest.raises(ValueError):
            mx.moe_unpermute_backward(*a, **kw)
