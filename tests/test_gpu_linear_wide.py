"""mx_linear_fused on more output features than one row of workgroups holds."""

import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mx_in", [False, True])
def test_linear_fused_2_28_features(mx_in):
    """Sums of small integers, exact in float32, against calls on the first and
    the last features alone."""
    K, N, n = 32, (1 << 28) + 34, 1000
    gen = torch.Generator(device="cuda").manual_seed(7)
    codes = torch.tensor([0, 0x38, 0xB8, 0x40, 0xC0], dtype=torch.uint8, device="cuda")   # 0, 1, -1, 2, -2
    w = torch.empty((N, K), dtype=torch.uint8, device="cuda")
    for i in range(0, N, 1 << 22):
        part = w[i:i + (1 << 22)]
        part.copy_(codes[torch.randint(0, 5, part.shape, dtype=torch.int32, device="cuda", generator=gen)])
    ws = torch.full((N, 1, 2), 127, dtype=torch.uint8, device="cuda")
    ws[:, 0, 1] = 0
    x = torch.randint(-2, 3, (1, K), device="cuda", generator=gen).bfloat16()
    xs = None
    if mx_in:
        x, xs = mx.mx_quantize(x)
    say(f"mx_linear_fused K={K} N={N} mx_in={mx_in}")
    y = mx.mx_linear_fused(x, w, ws, x_s=xs)
    first = mx.mx_linear_fused(x, w[:n], ws[:n], x_s=xs)
    last = mx.mx_linear_fused(x, w[N - n:], ws[N - n:], x_s=xs)
    mid = mx.mx_linear_fused(x, w[(1 << 27):(1 << 27) + n], ws[(1 << 27):(1 << 27) + n], x_s=xs)
    torch.cuda.synchronize()
    assert torch.equal(y[:, :n], first) and torch.equal(y[:, N - n:], last)
    assert torch.equal(y[:, (1 << 27):(1 << 27) + n], mid)


@pytest.mark.parametrize("T,K", [(1, 2048), (3, 544), (32, 2048), (32, 96)])
@pytest.mark.parametrize("N", [8192, 8193, 16424])
def test_few_bf16_tokens_around_a_round_of_workgroups(T, K, N):
    """Quantised by every workgroup itself up to 8192 features, ahead of the
    product past them: the product of mx_quantize's bytes either way.  Small
    integers, exact in float32 whatever the order of the sums."""
    gen = torch.Generator(device="cuda").manual_seed(T + N)
    x = torch.randint(-4, 5, (T, K), device="cuda", generator=gen).bfloat16()
    w, ws = mx.mx_quantize(torch.randint(-4, 5, (N, K), device="cuda", generator=gen).bfloat16())
    q, s = mx.mx_quantize(x)
    say(f"mx_linear_fused T={T} K={K} N={N} few bf16 tokens")
    a = mx.mx_linear_fused(x, w, ws)
    b = mx.mx_linear_fused(q, w, ws, x_s=s)
    aq, a_s = mx.mx_linear_fused(x, w, ws, act="relu", quantize_out=True)
    bq, b_s = mx.mx_linear_fused(q, w, ws, x_s=s, act="relu", quantize_out=True)
    torch.cuda.synchronize()
    want = (x.double() @ w_values(w, ws).T).bfloat16()
    assert torch.equal(a, want) and torch.equal(a, b) and torch.equal(aq, bq) and torch.equal(a_s, b_s)


def w_values(q, s):
    e = s.reshape(s.shape[0], -1)[:, : -(-q.shape[1] // 32)].double() - 127
    return q.view(torch.float8_e4m3fn).double() * torch.exp2(e).repeat_interleave(32, dim=1)[:, :q.shape[1]]


@pytest.mark.parametrize("T,K,N", [(7, 544, 640), (32, 2048, 8192), (33, 2080, 515), (600, 512, 4104), (1500, 672, 5633)])
def test_bf16_tokens_on_odd_addresses_and_in_place(T, K, N):
    """bf16 tokens that start at an odd element, with the residual in place:
    the bytes of the plain call."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, device="cuda", generator=gen).bfloat16()
    w, ws = mx.mx_quantize((0.05 * torch.randn(N, K, device="cuda", generator=gen)).bfloat16())
    res = torch.randn(T, N, device="cuda", generator=gen).bfloat16()
    say(f"mx_linear_fused T={T} K={K} N={N} odd bf16 tokens")
    want = mx.mx_linear_fused(x, w, ws, act="silu", residual=res)
    odd = torch.zeros(T * K + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, K)
    odd.copy_(x)
    r = torch.zeros(T * N + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, N)
    r.copy_(res)
    got = mx.mx_linear_fused(odd, w, ws, act="silu", residual=r, out=r)
    torch.cuda.synchronize()
    assert got is r and torch.equal(got, want)
