"""moe_permute on one-byte elements at any address: rows of odd widths and strides,
from an odd address to an odd address, through and past the caches."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import host, i32_dev, say
from oracle import int8_ref
from test_gpu_permute import routes

pytestmark = pytest.mark.gpu


SIZES = [
    (1, 1, 1, 1, 1), (9, 3, 5, 2, 4), (33, 15, 15, 3, 8), (33, 16, 17, 3, 8), (40, 17, 17, 8, 16), (300, 129, 131, 4, 32),
    (300, 2047, 2049, 2, 8), (3, 50001, 50003, 2, 5),
]
CASES = [(*s, offset) for s in SIZES for offset in (0, 1, 2, 3, 7)]
CASES += [(20000, 1001, 1003, 8, 64, offset) for offset in (0, 3)]   # over 128 MB: past the caches


@pytest.mark.parametrize("T,K,ld,k,E,offset", CASES)
def test_odd_bytes(T, K, ld, k, E, offset):
    gen = torch.Generator().manual_seed(T + offset)
    buf = torch.randint(-128, 128, (offset + T * ld,), generator=gen, dtype=torch.int8)
    x = buf[offset:].view(T, ld)[:, :K]
    on = torch.empty(offset + T * ld, dtype=torch.int8, device="cuda")
    on.copy_(buf)
    xs = torch.rand(T, generator=gen)
    ids = routes(T, k, E, T)
    M = T * k
    raw = torch.full((offset + M * K + 9,), 77, dtype=torch.int8, device="cuda")
    i32 = lambda: torch.empty(M, dtype=torch.int32, device="cuda")
    out = (raw[offset:offset + M * K].view(M, K), torch.empty(M, device="cuda"), i32(), i32(),
           torch.empty(E, dtype=torch.int64, device="cuda"))
    say(f"moe_permute int8 T={T} K={K} ld={ld} k={k} E={E} offset={offset}")
    got = mx.moe_permute(on[offset:].view(T, ld)[:, :K], i32_dev(ids), E, x_s=xs.cuda(), out=out)
    torch.cuda.synchronize()
    rows, sorted_row, eri, counts = int8_ref.permute_ref(x.numpy(), ids, E)
    assert np.array_equal(host(got[0]), rows)
    assert np.array_equal(host(got[1]), xs.numpy()[sorted_row // k])
    for a, b in zip(got[2:], (sorted_row, eri, counts)):
        assert np.array_equal(host(a), b)
    assert (raw[:offset] == 77).all() and (raw[offset + M * K:] == 77).all()


@pytest.mark.parametrize("dtype", [torch.uint8, torch.bool, torch.float8_e4m3fn])
def test_other_byte_types(dtype):
    T, K, k, E = 70, 33, 3, 9
    bits = torch.randint(0, 2 if dtype is torch.bool else 256, (T, K), dtype=torch.uint8)
    ids = routes(T, k, E, 4)
    got = mx.moe_permute(bits.view(dtype).cuda(), i32_dev(ids), E)
    torch.cuda.synchronize()
    assert got[0].dtype is dtype
    assert np.array_equal(host(got[0].view(torch.uint8)), int8_ref.permute_ref(bits.numpy(), ids, E)[0])
