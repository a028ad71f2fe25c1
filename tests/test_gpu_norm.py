"""mx_add_rmsnorm against the float64 definition.

Bound of the float32 arithmetic before the outputs' rounding, relative to n:
h = x + residual is rounded once (2^-24; the definition's h is exact, so the
bound is on |x| + |residual|, see `h_tol`).  The sum of squares adds positive
terms in a tree of at most 8 chunks in order x 4 + 6 lane steps + 16 waves and
two divisions' worth of roundings, each 2^-24 relative to a positive partial
sum: fewer than 40 steps, halved by the square root; rsqrt is within 2^-23 and
the two products within 2^-24 each.  Under 32 * 2^-24; rows over 65536 elements
add up to 16 more chunk steps at the lengths tested.  RTOL = 48 * 2^-24.
"""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from fused_util import F32_HALF, check_bf16, check_mx
from gpu_util import bf16_dev, bf16_host, f32_dev, guard_alloc, guards_intact, host, say
from oracle import fused_ref, mx_ref
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu
RTOL = 48 * F32_HALF
EPS = 1e-6


def rows_of(T, K, seed, scale=1.0):
    """bf16 bits: rows of different magnitudes, 1 % outlier channels, some
    zeros, the first row all zero when there are several."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, K)) * np.exp2(rng.integers(-8, 8, (T, 1))) * scale
    x[:, rng.permutation(K)[:-(-K // 100)]] *= 20
    x[rng.random((T, K)) < 0.02] = 0.0
    if T > 2:
        x[0] = 0.0
    return to_bf16_bits(x.astype(np.float32))


def make(T, K, residual, wf32, seed):
    x = rows_of(T, K, seed)
    r = rows_of(T, K, seed + 1, 2.0) if residual else None
    w = (1 + 0.2 * np.random.default_rng(seed + 2).standard_normal(K)).astype(np.float32)
    w_dev = f32_dev(w) if wf32 else bf16_dev(to_bf16_bits(w))
    w64 = w.astype(np.float64) if wf32 else mx_ref.bf16_to_f64(to_bf16_bits(w))
    return x, r, w_dev, w64


def check(got, x, r, w64, what, eps=EPS):
    q, s, r_out, y = got
    x64 = mx_ref.bf16_to_f64(x)
    r64 = None if r is None else mx_ref.bf16_to_f64(r)
    h, n = fused_ref.add_rmsnorm_ref(x64, r64, w64, eps)
    # the rounding of h where x and the residual cancel
    h_tol = F32_HALF * np.abs(h)
    scale = np.abs(w64) / np.sqrt((h * h).mean(axis=1) + eps)[:, None]
    if r_out is not None:
        check_bf16(mx_ref.bf16_to_f64(bf16_host(r_out)), h, F32_HALF, 0.0, what + " residual")
    if y is not None:
        check_bf16(mx_ref.bf16_to_f64(bf16_host(y)), n, RTOL, h_tol * scale, what + " y")
    if q is not None:
        check_mx(host(q), host(s), n, RTOL, h_tol * scale, what + " q")


SIZES = [(1, 1), (3, 7), (2, 31), (5, 32), (4, 33), (1, 64), (7, 100), (3, 512), (2, 513), (9, 520), (33, 1024),
         (65, 2048), (3, 2056), (5, 2049), (5, 4096), (2, 4304), (3, 8192), (2, 8200), (2, 16384), (1, 16391),
         (2, 32768), (1, 65536), (1, 65544), (2, 70001)]


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("residual,wf32", [(True, False), (False, True)])
def test_norm(T, K, residual, wf32):
    x, r, w, w64 = make(T, K, residual, wf32, 10 * T + K)
    say(f"mx_add_rmsnorm T={T} K={K} residual={residual} fp32 weight={wf32}")
    got = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r) if residual else None, EPS, norm_out=True)
    torch.cuda.synchronize()
    assert (got[2] is not None) == residual
    check(got, x, r, w64, f"T={T} K={K}")


def test_norm_many_rows():
    """More rows than the grid has workgroups: they walk the rows."""
    T, K = 40003, 64
    x, r, w, w64 = make(T, K, True, False, 3)
    say(f"mx_add_rmsnorm T={T} K={K}")
    got = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r), EPS, norm_out=True)
    torch.cuda.synchronize()
    check(got, x, r, w64, "many rows")


def test_norm_long_rows_walk():
    T, K = 600, 65601    # two-pass rows, more of them than the grid holds
    x, r, w, w64 = make(4, K, True, True, 4)
    x, r = np.tile(x, (T // 4, 1)), np.tile(r, (T // 4, 1))
    say(f"mx_add_rmsnorm T={T} K={K}")
    q, s, ro, y = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r), EPS, norm_out=True)
    torch.cuda.synchronize()
    check((q[:4], s[:4], ro[:4], y[:4]), x[:4], r[:4], w64, "long rows")
    for t in (q, s, ro, y):
        t = t.view(torch.uint8).view(T // 4, -1)
        assert bool((t == t[:1]).all())


@pytest.mark.parametrize("want", ["q", "y", "q+r", "y+r"])
def test_norm_chosen_outputs(want):
    """Outputs that are not asked for are not made; the others do not change."""
    T, K = 9, 520
    x, r, w, w64 = make(T, K, True, False, 5)
    full = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r), EPS, norm_out=True)
    out = [None] * 4
    if "q" in want:
        out[0], out[1] = torch.empty_like(full[0]), torch.empty_like(full[1])
    if "r" in want:
        out[2] = torch.empty_like(full[2])
    if "y" in want:
        out[3] = torch.empty_like(full[3])
    got = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r), EPS, out=tuple(out))
    torch.cuda.synchronize()
    for g, o, f in zip(got, out, full):
        assert g is o and (g is None or torch.equal(g, f))


@pytest.mark.parametrize("K,pad,off", [(512, 8, 0), (512, 3, 0), (511, 1, 1), (2048, 0, 1), (100, 28, 4), (8192, 8, 8)])
def test_norm_strides_and_alignments(K, pad, off):
    """Padded rows and buffers that start inside an allocation, guard bands
    around every output."""
    T = 5
    x, r, w, w64 = make(T, K, True, False, 6)
    def strided(bits):
        raw = torch.zeros(T * (K + pad) + off, dtype=torch.bfloat16, device="cuda")
        v = raw[off:].view(T, K + pad)[:, :K]
        v.copy_(bf16_dev(bits))
        return v
    raws = [guard_alloc(T * K + off, torch.uint8), guard_alloc(T * -(-K // 64) * 2, torch.uint8),
            guard_alloc(T * K + off, torch.bfloat16), guard_alloc(T * K + off, torch.bfloat16)]
    out = (raws[0][1][off:].view(T, K), raws[1][1].view(T, -1, 2), raws[2][1][off:].view(T, K),
           raws[3][1][off:].view(T, K))
    say(f"mx_add_rmsnorm strided K={K} pad={pad} offset={off}")
    got = mx.mx_add_rmsnorm(strided(x), w, strided(r), EPS, out=out)
    torch.cuda.synchronize()
    check(got, x, r, w64, "strided")
    for (raw, t), o in zip(raws, (off, 0, 2 * off, 2 * off)):
        assert guards_intact(raw, t.numel() * t.element_size())
        assert bool((raw[4096:4096 + o] == 0xA5).all())


@pytest.mark.parametrize("K", [96, 2048, 8200, 70001])
def test_norm_in_place(K):
    """residual_out over the residual, y over x: the same bytes."""
    T = 3
    x, r, w, _ = make(T, K, True, False, 7)
    full = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r), EPS, norm_out=True)
    xd, rd = bf16_dev(x), bf16_dev(r)
    q, s = torch.empty_like(full[0]), torch.empty_like(full[1])
    mx.mx_add_rmsnorm(xd, w, rd, EPS, out=(q, s, rd, xd))
    torch.cuda.synchronize()
    for g, f in zip((q, s, rd, xd), full):
        assert torch.equal(g, f)


def test_norm_leading_dims_and_empty():
    x, r, w, w64 = make(6, 100, True, False, 8)
    got = mx.mx_add_rmsnorm(bf16_dev(x).view(2, 3, 100), w, bf16_dev(r).view(2, 3, 100), EPS, norm_out=True)
    torch.cuda.synchronize()
    assert got[0].shape == (2, 3, 100) and got[1].shape == (2, 3, 2, 2)
    check([t.reshape((6,) + t.shape[2:]) for t in got], x, r, w64, "leading dims")
    q, s, ro, y = mx.mx_add_rmsnorm(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                                    torch.ones(64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 1, 2) and ro is None and y is None


def test_norm_large_eps_and_cancellation():
    """eps above the mean square; x and the residual cancelling to rounding size."""
    T, K = 4, 256
    x, r, w, w64 = make(T, K, True, True, 9)
    r = x ^ np.uint16(0x8000)
    r[:, ::7] = rows_of(T, K, 11, 2.0 ** -12)[:, ::7]
    for eps in (1e-6, 100.0):
        got = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r), eps, norm_out=True)
        torch.cuda.synchronize()
        check(got, x, r, w64, f"eps={eps}", eps)


def test_norm_offsets_past_32_bits():
    """The last rows of a batch of more than 2^32 elements."""
    K = 4096
    T = (1 << 32) // K + 5
    xs = rows_of(5, K, 12)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[-5:] = bf16_dev(xs)
    w = torch.ones(K, device="cuda")
    say(f"mx_add_rmsnorm T={T} K={K}")
    q, s, _, y = mx.mx_add_rmsnorm(x, w, eps=EPS, norm_out=True)
    torch.cuda.synchronize()
    check((q[-5:], s[-5:], None, y[-5:]), xs, None, np.ones(K), "past 2^32")
    assert not bool(q[:-5].view(torch.int64).any()) and not bool(s[:-5].any())


def test_norm_side_stream_and_graph():
    """On a side stream, and captured: every replay on new inputs against the
    eager call, with eager work between the replays."""
    T, K = 37, 2048
    sets = [make(T, K, True, False, 20 + i) for i in range(4)]
    xb, rb, w = bf16_dev(sets[0][0]), bf16_dev(sets[0][1]), sets[0][2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.mx_add_rmsnorm(xb, w, rb, EPS, norm_out=True, stream=side)
    side.synchronize()
    check(got, sets[0][0], sets[0][1], sets[0][3], "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = mx.mx_add_rmsnorm(xb, w, rb, EPS, norm_out=True)
    for i in (1, 2, 3):
        xb.copy_(bf16_dev(sets[i][0])); rb.copy_(bf16_dev(sets[i][1]))
        say(f"graph replay {i}")
        graph.replay()
        eager = mx.mx_add_rmsnorm(xb, w, rb, EPS, norm_out=True)
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b)
        check(outs, sets[i][0], sets[i][1], sets[0][3], f"replay {i}")
