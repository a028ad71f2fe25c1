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
