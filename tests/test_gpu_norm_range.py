"""mx_add_rmsnorm at the ends of its range: rows whose sum of squares, or mean
square, lies past fp32, and rows as long as it takes.  The definition, the
bound RTOL and the comparison are test_gpu_norm's; where the sum of squares
overflows, the reciprocal root is taken of the row scaled by a power of two,
which costs one rounding more when it comes out subnormal (root mean squares
over 2^126: at least 21 of its bits stay, 2^-22 or four of RTOL's 48 steps,
of which the bound there uses 32).

Rows of up to 2^24 elements: their squares go through 4 steps in a chunk of 8,
up to 42 additions of chunks, 6 of lanes and 15 of waves, the division and
eps: 69 roundings of positive partial sums, 2^-24 each at most, halved by the
root; with the root's own and the two products' less than 38 of RTOL's 48."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import bf16_dev, bf16_host, f32_dev, say
from oracle import mx_ref
from test_gpu_norm import EPS, RTOL, check, make, rows_of
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu


def large_rows(T, K, top, seed):
    """Rows around `top` beside ordinary and tiny ones, outliers and zeros in all."""
    x = mx_ref.bf16_to_f64(rows_of(T, K, seed))
    x *= (0.25 * top / np.maximum(np.abs(x).max(axis=1), 1e-30) * np.array([1.0, 2.0, 4.0])[np.arange(T) % 3])[:, None]
    x[1::4] = np.sign(x[1::4]) * top * 0.5                      # constant magnitude
    if T > 3:
        x[3] = mx_ref.bf16_to_f64(rows_of(1, K, seed + 9))[0]   # an ordinary row among them
    return to_bf16_bits(x.astype(np.float32))


# every plan of few rows, of many rows, and the two-pass one; aligned and not
PLANS = [(5, 512), (5, 2048), (5, 4096), (5, 8192), (5, 8190), (5, 16384), (2, 32768), (2, 65601),
         (300, 512), (300, 1024), (300, 2048), (300, 2041), (300, 4096), (300, 8192), (300, 16384), (300, 7)]


@pytest.mark.parametrize("T,K", PLANS)
@pytest.mark.parametrize("top", [1e18, 1e30, 1.5e38])
def test_norm_of_large_rows(T, K, top):
    x = large_rows(T, K, top, K)
    r = large_rows(T, K, top * 2.0 ** -10, K + 1) if K % 3 else None
    w = (1 + 0.2 * np.random.default_rng(K).standard_normal(K)).astype(np.float32)
    say(f"mx_add_rmsnorm large rows T={T} K={K} top={top}")
    got = mx.mx_add_rmsnorm(bf16_dev(x), f32_dev(w), None if r is None else bf16_dev(r), EPS, norm_out=True)
    torch.cuda.synchronize()
    check(got, x, r, w.astype(np.float64), f"T={T} K={K} top={top}")


def test_norm_of_large_rows_in_place():
    T, K = 300, 4096
    x, r = large_rows(T, K, 1e20, 1), large_rows(T, K, 1e19, 2)
    w = torch.ones(K, device="cuda")
    full = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r), EPS, norm_out=True)
    xd, rd = bf16_dev(x), bf16_dev(r)
    mx.mx_add_rmsnorm(xd, w, rd, EPS, out=(None, None, rd, xd))
    torch.cuda.synchronize()
    assert torch.equal(rd, full[2]) and torch.equal(xd, full[3])


def test_norm_of_large_rows_with_large_eps():
    """eps of the mean square's size beside it."""
    T, K = 5, 2048
    x = large_rows(T, K, 2e18, 3)
    for eps in (1e36, 3e38):
        got = mx.mx_add_rmsnorm(bf16_dev(x), torch.ones(K, device="cuda"), None, eps, norm_out=True)
        torch.cuda.synchronize()
        check(got, x, None, np.ones(K), f"eps={eps}", eps)


def tight(y, ref, rtol):
    """y is the rounding of a value within rtol of ref: nothing is added for it."""
    lo, hi = (mx_ref.f32_to_bf16((ref * f).astype(np.float32)) for f in (1 - rtol, 1 + rtol))
    return (y == lo) | (y == hi)


@pytest.mark.parametrize("K", [1 << 24, (1 << 24) - 5, (1 << 20) + 8])
def test_norm_of_the_longest_rows(K):
    x, r, w, w64 = make(1, K, True, True, K)
    say(f"mx_add_rmsnorm K={K}")
    got = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r), EPS, norm_out=True)
    torch.cuda.synchronize()
    check(got, x, r, w64, f"K={K}")


@pytest.mark.parametrize("a,b", [(1.0078125, 0.0017547607421875), (1.484375, 0.00127410888671875),
                                 (1.453125, 0.0247802734375)])
def test_norm_of_the_longest_rows_sum(a, b):
    """A row of one value whose square rounds the same way at nearly every step
    of a running sum (256 of RTOL's steps), beside weights that reach every
    rounding border of the output."""
    K = 1 << 24
    x, r = np.full((1, K), a, np.float32), np.full((1, K), b, np.float32)
    w = (1 + np.random.default_rng(1).random(K)).astype(np.float32)
    say(f"mx_add_rmsnorm K={K} of {a} + {b}")
    y = mx.mx_add_rmsnorm(bf16_dev(to_bf16_bits(x)), f32_dev(w), bf16_dev(to_bf16_bits(r)), EPS, quantize=False,
                          norm_out=True)[3]
    torch.cuda.synchronize()
    h = np.float64(np.float32(a) + np.float32(b))
    ref = h / np.sqrt(h * h + EPS) * w.astype(np.float64)
    bad = ~tight(bf16_host(y)[0], ref, RTOL)
    assert not bad.any(), (int(bad.sum()), ref[bad][:4], mx_ref.bf16_to_f64(bf16_host(y)[0][bad][:4]))
