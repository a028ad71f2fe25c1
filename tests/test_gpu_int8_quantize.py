"""int8_quantize: every code and scale equals the oracle's (the fp32 steps are
part of the definition, so nothing has to be bounded)."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import bf16_dev, guard_alloc, guards_intact, host, say
from oracle import int8_ref, mx_ref
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu


def draw(rows, K, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    x[:, rng.permutation(K)[:-(-K // 100)]] *= 20
    x[rng.random((rows, K)) < 0.02] = 0.0
    return to_bf16_bits(x.astype(np.float32))


def check(q, s, bits, what):
    rq, rs = int8_ref.int8_quantize_ref(mx_ref.bf16_to_f64(bits))
    assert np.array_equal(host(s), rs, equal_nan=True), (what, "scales")
    assert np.array_equal(host(q), rq), (what, "codes", np.argwhere(host(q) != rq)[:4].tolist())


SIZES = [
    (1, 1), (5, 3), (300, 7), (1, 8), (3, 9), (2, 15), (7, 64), (1, 511), (1, 512), (1, 513), (300, 500), (300, 520),
    (1, 2048), (300, 2048), (257, 2041), (2, 2056), (400, 2060), (1, 4096), (260, 4304), (1, 8192), (300, 8191), (1, 8200),
    (260, 8208), (1, 16384), (257, 16384), (2, 32768), (258, 32760), (1, 32776), (300, 33000), (1, 1 << 18), (2049, 1001),
]


@pytest.mark.parametrize("rows,K", SIZES)
def test_quantize(rows, K):
    xb = draw(rows, K, rows * 31 + K)
    raws = [guard_alloc(rows * K, torch.int8), guard_alloc(rows, torch.float32)]
    out = raws[0][1].view(rows, K), raws[1][1]
    say(f"int8_quantize rows={rows} K={K}")
    q, s = mx.int8_quantize(bf16_dev(xb), out=out)
    torch.cuda.synchronize()
    check(q, s, xb, "quantize")
    for raw, t in raws:
        assert guards_intact(raw, t.numel() * t.element_size())


def test_every_finite_value():
    """Each finite bf16 value beside amax = 127, 1 and the value itself."""
    v = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    v = v[(v & 0x7F80) != 0x7F80]
    one = to_bf16_bits(np.float32([1.0]))[0]
    for top in (to_bf16_bits(np.float32([127.0]))[0], one, 0):
        rows = np.stack([v, np.full_like(v, top)], axis=1)
        for x in (rows, np.repeat(rows, 8, axis=1)):   # rows of 2 and of 16 elements
            q, s = mx.int8_quantize(bf16_dev(x))
            torch.cuda.synchronize()
            check(q, s, x, f"top {top}")


def test_ties_and_the_floor():
    n = 4096
    x = np.zeros((6, n), np.float32)
    x[0] = (np.arange(n) % 255 - 127) / 2.0   # halves of the step
    x[0, 0] = 127.0
    x[1, 5] = 2.0 ** -133
    x[3] = -3.3895314e38
    x[4, 17] = 1.0
    x[5] = np.float32(2.0 ** -120) * (np.arange(n) % 3)
    xb = to_bf16_bits(x)
    q, s = mx.int8_quantize(bf16_dev(xb))
    torch.cuda.synchronize()
    check(q, s, xb, "edges")


@pytest.mark.parametrize("rows,K", [(9, 7), (9, 100), (9, 2048), (300, 2048), (9, 8000), (9, 30000), (9, 33000)])
def test_no_numbers(rows, K):
    """Rows with a NaN (of either sign, quiet or signalling), an infinity, both; the
    others as ever.  Products of such rows are NaN, also where the linear quantises."""
    xb = draw(rows, K, K)
    bad = {0: [0x7FC0], 1: [0xFF81], 2: [0x7F80], 3: [0xFF80], 5: [0x7F80, 0x7FFF], 6: [0xFFFF, 0xFF80]}
    for r, bits in bad.items():
        xb[r, [(r * 977 + 5 * i) % K for i in range(len(bits))]] = bits
    q, s = mx.int8_quantize(bf16_dev(xb))
    torch.cuda.synchronize()
    check(q, s, xb, "no numbers")
    assert not host(s)[sorted(set(range(9)) - set(bad))].max() == np.inf
    if K % 16 == 0:
        w, ws = mx.int8_quantize(torch.ones((40, K), dtype=torch.bfloat16, device="cuda"))
        y = mx.int8_linear(bf16_dev(xb), w, ws)
        assert torch.equal(y.isnan().all(dim=1), y.isnan().any(dim=1))
        assert torch.nonzero(y.isnan().any(dim=1)).flatten().tolist() == sorted(bad)


@pytest.mark.parametrize("K,ld,offset", [(2048, 2064, 0), (2048, 2049, 1), (100, 333, 3), (5, 9, 1), (33000, 33007, 1)])
def test_strided_rows(K, ld, offset):
    rows = 37
    xb = draw(rows, K, K + ld)
    buf = torch.full((rows * ld + offset,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = buf[offset:].view(rows, ld)[:, :K]
    x.copy_(bf16_dev(xb))
    q, s = mx.int8_quantize(x)
    torch.cuda.synchronize()
    check(q, s, xb, "strided")
    # codes on an odd address
    raw = torch.empty(rows * K + 1, dtype=torch.int8, device="cuda")
    q, s = mx.int8_quantize(x, out=(raw[1:].view(rows, K), s))
    torch.cuda.synchronize()
    check(q, s, xb, "odd address")


def test_leading_dims_and_empty():
    xb = draw(6 * 7, 96, 5)
    x = bf16_dev(xb).view(6, 7, 96)
    q, s = mx.int8_quantize(x)
    torch.cuda.synchronize()
    assert q.shape == (6, 7, 96) and s.shape == (6, 7)
    check(q.view(42, 96), s.view(42), xb, "3-D")
    q, s = mx.int8_quantize(x.transpose(0, 1))   # rows copied
    torch.cuda.synchronize()
    check(q.reshape(42, 96), s.reshape(42), np.ascontiguousarray(xb.reshape(6, 7, 96).swapaxes(0, 1)).reshape(42, 96), "transposed")
    q, s = mx.int8_quantize(bf16_dev(draw(1, 50, 2)).view(50))
    torch.cuda.synchronize()
    check(q.view(1, 50), s.view(1), draw(1, 50, 2), "1-D")
    q, s = mx.int8_quantize(x[:0])
    assert q.shape == (0, 7, 96) and s.shape == (0, 7)


def test_past_32_bits():
    """Rows whose codes and elements lie past 4 GiB."""
    rows, K = 70000, 65536
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    pick = [0, 32767, 32768, 65535, 65536, rows - 1]
    xb = draw(len(pick), K, 9)
    x[pick] = bf16_dev(xb)
    q, s = mx.int8_quantize(x)
    torch.cuda.synchronize()
    check(q[pick], s[pick], xb, "wide")
    assert int((q != 0).any(dim=1).sum()) == len(pick)
