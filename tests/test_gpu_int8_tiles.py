"""int8_linear's and gmm_int8's kernels by name: over several rounds of tiles, with
one, two, even, odd and incomplete k stages, tiles that end inside a fragment, and
the orders of loads and stores that only a full tile behind another one has.  The
queries say which kernel a size takes, so that a refit of the rule cannot move these
off the kernel they are for."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from fused_util import F32_HALF, check_bf16
from gpu_util import bf16_host, f32_dev, i64_dev, say
from oracle import int8_ref, mx_ref
from test_gpu_int8_products import codes, experts_case, i8_dev, linear_case, scales, swiglu_bound

pytestmark = pytest.mark.gpu

LINEAR = [   # kernel, T, K, N
    ("32x16", 5, 112, 70000), ("32x16", 16, 16, 33000), ("32x16", 16, 400, 33000), ("32x16", 13, 256, 40000),
    ("32x16 wide", 5, 1040, 4100), ("32x16 wide", 16, 2064, 97), ("32x16 wide", 1, 4096, 8192), ("32x16 wide", 100, 1040, 1030),
    ("32x32", 30, 400, 70000), ("32x32", 60, 1040, 12300), ("32x32", 30, 256, 33000), ("32x32", 200, 256, 2050),
    ("48x48", 40, 112, 70000), ("48x48", 40, 400, 70000), ("48x48", 333, 1040, 2050), ("48x48", 40, 16, 70000), ("48x48", 100, 256, 4100),
    ("64x64", 60, 208, 70000), ("64x64", 60, 1040, 70000), ("64x64", 2900, 112, 515), ("64x64", 2900, 256, 515),
    ("128x128", 1500, 112, 12300), ("128x128", 4300, 128, 4100), ("128x128", 4300, 208, 4100), ("128x128", 1500, 400, 12300),
    ("128x128", 333, 256, 8200), ("256x256", 2900, 112, 4100), ("256x256", 2900, 128, 4100), ("256x256", 2900, 256, 4100),
    ("256x256", 2900, 400, 4100), ("256x256", 8100, 272, 4090), ("256x256", 8192, 128, 4096),
]


@pytest.mark.parametrize("i", range(len(LINEAR)))
def test_linear(i):
    kernel, T, K, N = LINEAR[i]
    assert mx.int8_linear_kernel(T, K, N, True) == kernel
    linear_case(T, K, N, 900 + i, bias=["none", "bf16", "fp32"][i % 3], act=["none", "silu", "gelu_tanh", "relu"][i % 4],
                residual=i % 2 == 0, in_place=i % 4 == 0, what=kernel)


EXPERTS = [   # kernel, swiglu, rows per expert, K, N
    ("32x16", 0, [3] * 40, 112, 2050), ("32x16", 0, [17] * 8, 128, 1030), ("32x16", 1, [3, 0, 5, 1] * 10, 256, 1030),
    ("32x16", 1, [1] * 40, 16, 200), ("32x16 wide", 0, [17] * 8, 1040, 515), ("32x16 wide", 1, [1] * 8, 1040, 515),
    ("32x32", 0, [17] * 40, 400, 1030), ("32x32", 0, [17] * 8, 1040, 4100), ("32x32", 1, [17, 33, 1, 16] * 2, 208, 4100),
    ("32x32", 1, [130] * 8, 208, 200), ("64x64", 0, [17] * 40, 208, 2050), ("64x64", 0, [17] * 40, 256, 2050),
    ("64x64", 1, [20, 17, 0, 31] * 10, 256, 1030), ("64x64", 1, [17] * 40, 256, 1024), ("128x128", 0, [60, 61, 0, 119] * 10, 112, 4100),
    ("128x128", 0, [130] * 8, 128, 4096), ("128x128", 0, [60] * 40, 256, 4100), ("128x128", 1, [130] * 8, 112, 4100),
    ("128x128", 1, [128] * 8, 128, 2048), ("128x128", 1, [60] * 40, 256, 1030), ("256x256", 0, [300] * 8, 128, 4100),
    ("256x256", 0, [130] * 40, 112, 2050), ("256x256", 0, [256, 300, 212, 257] * 10, 400, 1024), ("256x256", 1, [300] * 8, 128, 4100),
    ("256x256", 1, [256] * 8, 128, 4096), ("256x256", 1, [256] * 12, 256, 4096), ("256x256", 1, [256, 512, 0, 300] * 4, 384, 2048),
    ("256x256", 1, [130] * 40, 112, 2050), ("256x256", 1, [512, 511, 513], 640, 6400), ("256x256", 1, [700] * 3, 16, 4100),
]


@pytest.mark.parametrize("i", range(len(EXPERTS)))
def test_experts(i):
    kernel, swiglu, counts, K, N = EXPERTS[i]
    assert mx.gmm_int8_kernel(sum(counts), N, K, len(counts), swiglu) == kernel
    experts_case(counts, K, N, bool(swiglu), 700 + i, kind=i % 2, what=kernel)


@pytest.mark.parametrize("swiglu", [0, 1])
@pytest.mark.parametrize("kernel,M,K,N,E", [
    ("32x16", 64, 256, 64, 1024), ("64x64", 2000, 256, 512, 64), ("128x128", 4000, 256, 512, 64), ("256x256", 16000, 256, 512, 64),
])
def test_uneven_experts(kernel, M, K, N, E, swiglu):
    """The host chooses for even experts; the device's list may say anything: all rows
    with one expert, with the last one, most of them with nobody."""
    if swiglu:
        N //= 2
    assert mx.gmm_int8_kernel(M, N, K, E, swiglu) == kernel
    rng = np.random.default_rng(E + M)
    rows = 2 * N if swiglu else N
    a, a_s, ws = codes(rng, (M, K)), scales(rng, M, 1.0), scales(rng, (E, rows), 3 / (40 * 40 * np.sqrt(K)))
    w = codes(rng, (E, rows, K))
    ad, asd, wd, wsd = i8_dev(a), f32_dev(a_s), i8_dev(w), f32_dev(ws)
    for pick in ([(0, M)], [(E - 1, M)], [(E // 2, 1)], [(1, M // 2 + 1), (E - 1, M // 3)]):
        counts = np.zeros(E, np.int64)
        for e, n in pick:
            counts[e] = n
        say(f"gmm_int8 uneven {kernel} {pick}")
        out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
        mx.gmm_int8(ad, asd, wd, wsd, i64_dev(counts), swiglu=bool(swiglu), out=out)
        torch.cuda.synchronize()
        n = int(counts.sum())
        ref, gu = int8_ref.gmm_int8_ref(a[:n], a_s[:n], w, ws, counts, bool(swiglu))
        err = swiglu_bound(ref, gu) if swiglu else 3.01 * F32_HALF * np.abs(ref)
        check_bf16(mx_ref.bf16_to_f64(bf16_host(out[:n])), ref, 0.0, err, str(pick))
        assert (out[n:] == 3).all()


def test_queries():
    assert mx.int8_linear_kernel(1, 2048, 4096, False) == "32x16 bf16"
    for call in (lambda: mx.int8_linear_kernel(0, 64, 64, True), lambda: mx.int8_linear_kernel(4, 24, 64, True),
                 lambda: mx.gmm_int8_kernel(0, 64, 64, 4), lambda: mx.gmm_int8_kernel(4, 64, 64, 1025)):
        with pytest.raises(mx.MxError):
            call()
