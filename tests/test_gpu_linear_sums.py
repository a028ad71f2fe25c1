"""What mx_linear_fused's sums keep, as its contract says: of 8 consecutive k
each product is truncated to a multiple of 2^(e - 13), e the largest of their
sums of operand exponents, and everything else adds in float32.

Every case plants one product of +-2^14 and one of 7 (e = 14: multiples of 2)
in a row of zeros and takes the large one off again with the residual, which is
exact: float32 holds 2^14 + 7."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import bf16_dev, bf16_host, say, u8_dev
from oracle import mx_ref
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel,T,N,K", [("32x32", 96, 34, 96), ("64x64 twice per CU", 132, 5493, 64),
                                          ("128x128", 450, 4104, 64), ("256x256", 1440, 5640, 160)])
@pytest.mark.parametrize("big_at", [0, 5, 31, 45])
def test_products_beside_a_large_one(kernel, T, N, K, big_at):
    assert mx.linear_fused_kernel(T, K, N, True) == kernel
    small_at = (big_at + 1 + np.arange(T) % (K - 1)) % K   # token t's; never big_at
    x, w = np.zeros((T, K)), np.ones((N, K))
    sign = np.where(np.arange(T) // (K - 1) % 2, -1.0, 1.0)
    x[:, big_at] = 128.0 * sign
    x[np.arange(T), small_at] = 7.0
    w[:, big_at] = 128.0
    x[T - 1] = 0.0
    one = lambda rows: np.full((rows, -(-K // 64), 2), 127, np.uint8)
    xs, ws = one(T), one(N)
    if K // 32 % 2:
        xs[:, -1, 1] = ws[:, -1, 1] = 0
    res = np.repeat(-x[:, big_at:big_at + 1] * 128.0, N, axis=1)
    say(f"mx_linear_fused {kernel} T={T} K={K} N={N} large product at {big_at}")
    y = mx.mx_linear_fused(u8_dev(mx_ref.e4m3_encode(x)), u8_dev(mx_ref.e4m3_encode(w)), u8_dev(ws), x_s=u8_dev(xs),
                           residual=bf16_dev(to_bf16_bits(res.astype(np.float32))))
    torch.cuda.synchronize()
    y = mx_ref.bf16_to_f64(bf16_host(y))
    want = np.full((T, 1), 7.0); want[T - 1] = 0.0
    same_group = (small_at // 8 == big_at // 8)[:, None]
    off = np.abs(y - want)
    assert (off[~same_group[:, 0]] == 0).all()
    assert (off < 2.0).all() and ((y == 6.0) | (y == 7.0) | (y == 8.0) | (want == 0)).all()
