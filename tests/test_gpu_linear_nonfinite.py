"""Tokens, channels and biases that are no numbers come out of a linear's epilogue
as NaN, whatever the activation (relu among them), in every kernel; everything
beside them keeps its bits."""

import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import say

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
NAN, INF = float("nan"), float("inf")

INT8 = [   # kernel, T, K, N, x is int8
    ("32x16 bf16", 5, 528, 257, False), ("32x16 bf16", 16, 1024, 1030, False), ("32x16", 16, 400, 33000, True),
    ("32x16 wide", 16, 2064, 97, True), ("32x32", 200, 256, 2050, True), ("48x48", 333, 1040, 2050, True),
    ("64x64", 2900, 112, 515, True), ("128x128", 333, 256, 8200, True), ("128x128", 333, 256, 8200, False),
    ("256x256", 2900, 272, 4100, True), ("256x256", 2900, 272, 4100, False),
]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("kernel,T,K,N,int8_in", INT8)
def test_int8_linear(kernel, T, K, N, int8_in, residual):
    assert mx.int8_linear_kernel(T, K, N, int8_in) == kernel
    gen = torch.Generator(device="cuda").manual_seed(T + N)
    x = torch.randn((T, K), generator=gen, device="cuda").bfloat16()
    w, ws = mx.int8_quantize(torch.randn((N, K), generator=gen, device="cuda").bfloat16())
    b = torch.randn(N, generator=gen, device="cuda")
    res = torch.randn((T, N), generator=gen, device="cuda").bfloat16() if residual else None
    bad_x, bad_ws, bad_b = x.clone(), ws.clone(), b.clone()
    bad_x[0, K // 2], bad_x[T // 2, 0], bad_x[T - 1, K - 1] = NAN, INF, -INF
    bad_ws[1], bad_ws[N - 2], bad_b[N // 2], bad_b[N - 1] = NAN, INF, NAN, -NAN
    rows, cols = [0, T // 2, T - 1], [1, N // 2, N - 1]
    if not int8_in:
        call = lambda x, ws, b, act: mx.int8_linear(x, w, ws, bias=b, act=act, residual=res)
    else:
        def call(x, ws, b, act):
            q, s = mx.int8_quantize(x)
            return mx.int8_linear(q, w, ws, x_s=s, bias=b, act=act, residual=res)
    for act in ACTS:
        say(f"int8_linear {kernel} T={T} K={K} N={N} int8_in={int8_in} act={act} residual={residual}")
        good, got = call(x, ws, b, act), call(bad_x, bad_ws, bad_b, act)
        torch.cuda.synchronize()
        none = torch.zeros((T, N), dtype=torch.bool, device="cuda")
        none[rows] = True
        none[:, cols] = True
        none[:, N - 2] |= got[:, N - 2].isnan()   # (an infinite channel: any of infinity, NaN and an activation's 0)
        assert torch.equal(got.isnan(), none), (act, torch.nonzero(got.isnan() != none)[:4].tolist())
        none[:, N - 2] = True
        assert torch.equal(got[~none], good[~none]), act


MX = [   # kernel, T, K, N
    ("32x32 bf16", 7, 544, 640), ("32x32", 40, 2080, 515), ("128x128", 450, 256, 4104), ("256x256", 1440, 512, 5640),
]


@pytest.mark.parametrize("kernel,T,K,N", MX)
def test_mx_linear_fused(kernel, T, K, N):
    """The same epilogue: a bias that is no number is not hidden."""
    mx_in = kernel != "32x32 bf16"
    assert mx.linear_fused_kernel(T, K, N, mx_in) == kernel
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, K), generator=gen, device="cuda").bfloat16()
    w, ws = mx.mx_quantize(torch.randn((N, K), generator=gen, device="cuda").bfloat16())
    x, xs = mx.mx_quantize(x) if mx_in else (x, None)
    b = torch.randn(N, generator=gen, device="cuda")
    bad = b.clone()
    bad[2], bad[N - 1] = NAN, NAN
    for act in ACTS:
        say(f"mx_linear_fused {kernel} T={T} K={K} N={N} act={act}")
        good, got = (mx.mx_linear_fused(x, w, ws, x_s=xs, bias=v, act=act) for v in (b, bad))
        torch.cuda.synchronize()
        none = torch.zeros((T, N), dtype=torch.bool, device="cuda")
        none[:, [2, N - 1]] = True
        assert torch.equal(got.isnan(), none), act
        assert torch.equal(got[~none], good[~none]), act
