"""mx_linear_fused against the float64 definition.

Bound of the arithmetic before the outputs' rounding.  The matrix instruction
takes the 64 products of its step in aligned groups of 8 consecutive k: within
a group each product is truncated to a multiple of 2^(e - 13), e the largest of
the group's sums of operand exponents (a payload below 2^-6, zero too, counts
with exponent -6).  Planting one large product beside one small one at every
position shows it: 1.75 * 2^2 beside 2^14 comes out as 6, and the same product
outside the group of 8 exact to 24 bits.  So a group is off by less than 8 *
2^-13 max P(x) P(w), P(v) = max(|payload|, 2^-6) in its block's scale.  The
groups, steps and partial sums then add in float32: with A = sum_k |x_k w_k|
every partial sum is at most A, and the steps, at most 16 partial sums, the
bias and the two terms of the epilogue cost (K / 64 + 20) 2^-22 A.

The activations' slopes stay under 1.13.  Their own error is relative: the
hardware exp of an argument a is within (|a| + 2) 2^-23, reciprocal and
products within 2^-23 each; |a| is |z| for silu, at most z^2 / 2 + 2 for gelu,
and 2 |u| <= 1.6 |z| (1 + 0.045 z^2) for gelu_tanh: (z^2 + 4 |z| + 16) 2^-23
(1 + 0.1 |z|) covers the three.
"""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from fused_util import F32_HALF, check_bf16, check_mx
from gpu_util import bf16_dev, bf16_host, f32_dev, guard_alloc, guards_intact, host, say, u8_dev
from oracle import fused_ref, mx_ref
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def draw(T, K, N, seed, scale=0.05):
    """bf16 token rows of different magnitudes with outlier channels, and MXFP8
    weights, as bits and as values."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, K)) * np.exp2(rng.integers(-3, 3, (T, 1)))
    x[:, rng.permutation(K)[:-(-K // 100)]] *= 20
    x[rng.random((T, K)) < 0.02] = 0.0
    xb = to_bf16_bits(x.astype(np.float32))
    w = to_bf16_bits((rng.standard_normal((N, K)) * scale).astype(np.float32))
    return xb, mx_ref.mx_quantize_ref(mx_ref.bf16_to_f64(xb)), mx_ref.mx_quantize_ref(mx_ref.bf16_to_f64(w))


def group_maxima(xq, wq):
    """Sum over the groups of 8 consecutive k of max P(x) P(w), [T, N]."""
    def p_of(q, s):
        K = q.shape[1]
        pay = np.maximum(np.abs(mx_ref.e4m3_decode(q)), 2.0 ** -6)
        e = mx_ref.scales_flat(s, K).astype(np.float64) - 127
        return torch.from_numpy((pay * np.repeat(np.exp2(e), 32, axis=1)[:, :K]).astype(np.float32)).cuda()
    px, pw = p_of(*xq), p_of(*wq)
    total = torch.zeros(px.shape[0], pw.shape[0], device="cuda")
    for g in range(0, px.shape[1], 8):
        best = px[:, g, None] * pw[None, :, g]
        for k in range(g + 1, g + 8):
            torch.maximum(best, px[:, k, None] * pw[None, :, k], out=best)
        total += best
    return total.double().cpu().numpy() * (1 + 2.0 ** -12)   # these sums are float32


def reference(xq, wq, bias, act, res):
    """(out, its float32 error bound), float64."""
    x, w = mx_ref.mx_dequantize_ref(*xq), mx_ref.mx_dequantize_ref(*wq)
    K = x.shape[1]
    z = x @ w.T
    zerr = (K / 64 + 20) * 2.0 ** -22 * (np.abs(x) @ np.abs(w).T) + 2.0 ** -10 * group_maxima(xq, wq)
    if bias is not None:
        z = z + bias
        zerr = zerr + F32_HALF * np.abs(z)
    a = fused_ref.activate_ref(z, act)
    err = 1.13 * zerr
    if act not in ("none", "relu"):
        err = err + (z * z + 4 * np.abs(z) + 16) * (1 + 0.1 * np.abs(z)) * 2.0 ** -23 * np.abs(a) + 1e-37
    out = a if res is None else a + res
    return out, err + F32_HALF * (np.abs(out) + err)


def run_case(T, K, N, seed, mx_in, bias, act, residual, mx_out, what):
    xb, xq, wq = draw(T, K, N, seed)
    rng = np.random.default_rng(seed + 1)
    b = rng.standard_normal(N).astype(np.float32)
    bd, b64 = None, None
    if bias == "f32":
        bd, b64 = f32_dev(b), b.astype(np.float64)
    elif bias == "bf16":
        bd, b64 = bf16_dev(to_bf16_bits(b)), mx_ref.bf16_to_f64(to_bf16_bits(b))
    rb = to_bf16_bits((2 * rng.standard_normal((T, N))).astype(np.float32)) if residual else None
    r64 = mx_ref.bf16_to_f64(rb) if residual else None
    say(f"mx_linear_fused {what} T={T} K={K} N={N} mx_in={mx_in} bias={bias} act={act} residual={residual} mx_out={mx_out}")
    x, xs = (u8_dev(xq[0]), u8_dev(xq[1])) if mx_in else (bf16_dev(xb), None)
    if mx_out:
        raws = [guard_alloc(T * N, torch.uint8), guard_alloc(T * -(-N // 64) * 2, torch.uint8)]
        out = (raws[0][1].view(T, N), raws[1][1].view(T, -1, 2))
    else:
        raws = [guard_alloc(T * N, torch.bfloat16)]
        out = raws[0][1].view(T, N)
    got = mx.mx_linear_fused(x, u8_dev(wq[0]), u8_dev(wq[1]), x_s=xs, bias=bd, act=act,
                             residual=bf16_dev(rb) if residual else None, out=out)
    torch.cuda.synchronize()
    for raw, t in raws:
        assert guards_intact(raw, t.numel() * t.element_size()), what
    ref, err = reference(xq, wq, b64, act, r64)
    if mx_out:
        check_mx(host(got[0]), host(got[1]), ref, 0.0, err, what)
    else:
        check_bf16(mx_ref.bf16_to_f64(bf16_host(got)), ref, 0.0, err, what)


SIZES = [
    (1, 32, 1), (1, 128, 64), (2, 64, 33), (1, 2048, 2048), (3, 96, 257), (8, 1024, 100), (9, 160, 31), (16, 2080, 255),
    (17, 384, 1000), (31, 4096, 96), (32, 224, 512), (32, 8192, 70), (33, 128, 64), (64, 256, 129), (65, 1024, 200),
    (127, 288, 65), (128, 2048, 256), (203, 2080, 515), (257, 384, 768), (300, 32, 300), (520, 4096, 192),
    (1100, 544, 1030), (2049, 256, 264),
]


@pytest.mark.parametrize("i", range(len(SIZES)))
def test_linear_fused(i):
    """Every size with two of the epilogues, all of which come up."""
    T, K, N = SIZES[i]
    for j in (0, 1):
        c = 2 * i + j
        run_case(T, K, N, 100 + c, mx_in=c % 3 != 0, bias=["none", "bf16", "f32"][c % 3], act=ACTS[c % 5],
                 residual=c % 4 < 2, mx_out=j == 1, what=f"case {c}")


# two sizes or more, with an incomplete last k stage and without, for each tile
# shape that only wide outputs reach (weight rows x tokens), and for 32 x 32
# tiles over more than one round
WIDE = [
    (45, 96, 4225), (128, 640, 4096),        # 32 x 32
    (7, 160, 8300), (13, 512, 9000),         # 32 x 32, few tokens
    (131, 992, 5505), (129, 896, 5633),      # 32 x 32, two rounds
    (100, 1056, 4099), (150, 512, 5440),     # 64 x 64
    (161, 1056, 5700), (288, 640, 5400),     # 64 x 96
    (199, 160, 4130), (330, 384, 4810),      # 64 x 64, two workgroups per CU
    (450, 416, 4100), (600, 768, 4500),      # 128 x 128
    (1030, 1696, 4099), (1030, 1664, 4096),  # 256 x 128
    (1440, 672, 5633), (1500, 1280, 5633),   # 256 x 256
]


@pytest.mark.parametrize("i", range(len(WIDE)))
def test_linear_fused_wide(i):
    T, K, N = WIDE[i]
    run_case(T, K, N, 200 + i, mx_in=i % 3 != 0, bias=["none", "bf16", "f32"][i % 3], act=ACTS[i % 5],
             residual=i % 4 < 2, mx_out=i % 7 == 3, what=f"wide {i}")
    exact_case(T, K, N)


@pytest.mark.parametrize("T", [5, 200, 600])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("mx_out", [False, True])
def test_linear_fused_epilogues(T, act, mx_out):
    run_case(T, 256, 320, T, True, "f32", act, True, mx_out, "epilogue")


def exact_case(T, K, N):
    """Small integers with power-of-two scales: every sum is exact in float32,
    so the bf16 output is the correctly rounded one, at every tile position."""
    rng = np.random.default_rng(T)
    # scales near 1 keep every product a small integer times 2^-3
    xi = rng.integers(-15, 16, (T, K)).astype(np.float64)
    wi = rng.integers(-15, 16, (N, K)).astype(np.float64)
    xq, wq = mx_ref.e4m3_encode(xi), mx_ref.e4m3_encode(wi)
    nb = -(-K // 32)
    pad = -(-K // 64) * 2
    xs, ws = np.zeros((T, pad), np.uint8), np.zeros((N, pad), np.uint8)
    xs[:, :nb] = rng.integers(125, 129, (T, nb))
    ws[:, :nb] = rng.integers(126, 129, (N, nb))
    xs, ws = xs.reshape(T, -1, 2), ws.reshape(N, -1, 2)
    say(f"mx_linear_fused exact T={T} K={K} N={N}")
    y = mx.mx_linear_fused(u8_dev(xq), u8_dev(wq), u8_dev(ws), x_s=u8_dev(xs))
    torch.cuda.synchronize()
    z = mx_ref.mx_dequantize_ref(xq, xs) @ mx_ref.mx_dequantize_ref(wq, ws).T
    assert np.abs(z).max() < 2 ** 19   # 24 bits from the unit 2^-3
    assert np.array_equal(bf16_host(y), mx_ref.f32_to_bf16(z.astype(np.float32)))


@pytest.mark.parametrize("T,K,N", [(1, 128, 96), (29, 416, 131), (64, 1024, 256), (300, 640, 520), (1030, 256, 1030)])
def test_linear_fused_exact(T, K, N):
    exact_case(T, K, N)


def test_linear_fused_quantised_input_is_mx_quantize():
    """bf16 input gives the bytes of mx_quantize's output as input."""
    for T in (1, 20, 130):
        xb, _, wq = draw(T, 640, 160, T)
        x = bf16_dev(xb)
        q, s = mx.mx_quantize(x)
        a = mx.mx_linear_fused(x, u8_dev(wq[0]), u8_dev(wq[1]), act="silu")
        b = mx.mx_linear_fused(q, u8_dev(wq[0]), u8_dev(wq[1]), x_s=s, act="silu")
        torch.cuda.synchronize()
        assert torch.equal(a, b), T


def test_linear_fused_zero_and_large_values():
    """All-zero tokens and weights (scale byte 0 throughout), the largest block
    scales, and an activation far into both tails."""
    T, K, N = 40, 128, 64
    z8, s8 = np.zeros((T, K), np.uint8), np.zeros((T, 2, 2), np.uint8)
    wq, ws = np.zeros((N, K), np.uint8), np.zeros((N, 2, 2), np.uint8)
    q, s = mx.mx_linear_fused(u8_dev(z8), u8_dev(wq), u8_dev(ws), x_s=u8_dev(s8), quantize_out=True)
    torch.cuda.synchronize()
    assert not host(q).any() and not host(s).any()
    xq = mx_ref.mx_quantize_ref(np.full((T, K), 448.0 * 2.0 ** 40))
    w = np.zeros((N, K)); w[:, 0] = np.where(np.arange(N) % 2, 1.0, -1.0)
    wqr = mx_ref.mx_quantize_ref(w)
    for act in ACTS:
        y = mx.mx_linear_fused(u8_dev(xq[0]), u8_dev(wqr[0]), u8_dev(wqr[1]), x_s=u8_dev(xq[1]), act=act)
        torch.cuda.synchronize()
        big = 448.0 * 2.0 ** 40
        want = np.where(np.arange(N) % 2, big, -big if act == "none" else 0.0)
        got = mx_ref.bf16_to_f64(bf16_host(y))
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want)), act


@pytest.mark.parametrize("T,N", [(4, 100), (100, 256), (700, 512)])
def test_linear_fused_residual_in_place(T, N):
    xb, xq, wq = draw(T, 256, N, 7)
    rb = to_bf16_bits(np.random.default_rng(8).standard_normal((T, N)).astype(np.float32))
    args = (u8_dev(xq[0]), u8_dev(wq[0]), u8_dev(wq[1]))
    want = mx.mx_linear_fused(*args, x_s=u8_dev(xq[1]), residual=bf16_dev(rb))
    r = bf16_dev(rb)
    got = mx.mx_linear_fused(*args, x_s=u8_dev(xq[1]), residual=r, out=r)
    torch.cuda.synchronize()
    assert got is r and torch.equal(got, want)


@pytest.mark.parametrize("T", [3, 70, 600])
def test_linear_fused_unaligned_rows(T):
    """Residual and outputs that start at odd elements; odd and even widths."""
    for N in (63, 64, 256):
        xb, xq, wq = draw(T, 128, N, 9 + N)
        args = (u8_dev(xq[0]), u8_dev(wq[0]), u8_dev(wq[1]))
        rb = to_bf16_bits(np.random.default_rng(9).standard_normal((T, N)).astype(np.float32))
        want = mx.mx_linear_fused(*args, x_s=u8_dev(xq[1]), residual=bf16_dev(rb))
        wq8, ws8 = mx.mx_linear_fused(*args, x_s=u8_dev(xq[1]), residual=bf16_dev(rb), quantize_out=True)
        off = lambda n, dt: torch.empty(n + 1, dtype=dt, device="cuda")[1:]
        r = off(T * N, torch.bfloat16).view(T, N); r.copy_(bf16_dev(rb))
        y = mx.mx_linear_fused(*args, x_s=u8_dev(xq[1]), residual=r, out=off(T * N, torch.bfloat16).view(T, N))
        q, s = mx.mx_linear_fused(*args, x_s=u8_dev(xq[1]), residual=r,
                                  out=(off(T * N, torch.uint8).view(T, N), off(ws8.numel(), torch.uint8).view(ws8.shape)))
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(q, wq8) and torch.equal(s, ws8), N


def test_linear_fused_rows_do_not_depend_on_the_batch():
    """A token's output within one kernel's range is the same bytes in any
    batch and position."""
    T = 600
    xb, xq, wq = draw(T, 512, 384, 10)
    x, xs, w, ws = u8_dev(xq[0]), u8_dev(xq[1]), u8_dev(wq[0]), u8_dev(wq[1])
    full = mx.mx_linear_fused(x, w, ws, x_s=xs, act="silu")
    again = mx.mx_linear_fused(x, w, ws, x_s=xs, act="silu")
    rolled = mx.mx_linear_fused(x.roll(77, 0), w, ws, x_s=xs.roll(77, 0), act="silu")
    torch.cuda.synchronize()
    assert torch.equal(full, again) and torch.equal(rolled, full.roll(77, 0))


def test_linear_fused_empty():
    y = mx.mx_linear_fused(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"),
                           torch.zeros((100, 128), dtype=torch.uint8, device="cuda"),
                           torch.zeros((100, 2, 2), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert y.shape == (0, 100)


@pytest.mark.parametrize("T", [2, 150, 1030])
def test_linear_fused_stream_and_graph(T):
    """On a side stream, and captured with its workspace shared by two graphs:
    every replay on new tokens against the eager call."""
    K, N = 512, 260
    sets = [draw(T, K, N, 40 + i) for i in range(4)]
    w, ws = u8_dev(sets[0][2][0]), u8_dev(sets[0][2][1])
    bufs = [bf16_dev(sets[0][0]) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.mx_linear_fused(bufs[0], w, ws, stream=side)
    side.synchronize()
    assert torch.equal(got, mx.mx_linear_fused(bufs[0], w, ws))
    space = torch.empty(max(256, mx.linear_fused_workspace_size(T, K, N, False)), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mx.mx_linear_fused(b, w, ws, act="gelu", workspace=space))
        graphs.append(g)
    for i in range(1, 4):
        for j in (0, 1):
            bufs[j].copy_(bf16_dev(sets[(i + j) % 4][0]))
            say(f"replay {i} of graph {j}")
            graphs[j].replay()
            eager = mx.mx_linear_fused(bufs[j], w, ws, act="gelu")
            torch.cuda.synchronize()
            assert torch.equal(outs[j], eager), (i, j)


@pytest.mark.parametrize("T,K,N,act", [
    (32, 2048, 96, "none"), (16, 4096, 130, "silu"), (1, 65536, 33, "none"), (31, 2080, 64, "gelu"),
    (32, 2080, 64, "none"), (7, 96, 1000, "relu"), (2, 32736, 40, "none"), (32, 32, 32, "gelu_tanh"),
])
def test_linear_fused_few_bf16_tokens(T, K, N, act):
    """bf16 tokens on both sides of the size that workgroups quantise for
    themselves (T <= 32, T K <= 65536, no workspace): the bytes of the MXFP8 call
    on mx_quantize's output wherever the same kernel runs, and the definition's."""
    assert (mx.linear_fused_workspace_size(T, K, N, False) == 0) == (T * K <= 65536)
    run_case(T, K, N, T + K, False, "f32", act, True, False, "few bf16")
    run_case(T, K, N, T + K + 1, False, "none", act, False, True, "few bf16")
    xb, _, wq = draw(T, K, N, 3)
    x = bf16_dev(xb)
    raw = torch.zeros(T * K + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, K)   # an odd address
    raw.copy_(x)
    a = mx.mx_linear_fused(x, u8_dev(wq[0]), u8_dev(wq[1]), act=act)
    b = mx.mx_linear_fused(raw, u8_dev(wq[0]), u8_dev(wq[1]), act=act)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,K,N", [(600000, 32, 4104), (300, 32768, 140000), (2, 32768, 140003), ((1 << 26) + 32, 64, 3)])
def test_linear_fused_offsets_past_32_bits(T, K, N):
    """The last rows and features of operands and outputs over 4 GiB, against
    the same ones in a call of their own: sums of small integers, exact in
    float32 in any order."""
    say(f"mx_linear_fused past 32 bits T={T} K={K} N={N}")
    gen = torch.Generator(device="cuda").manual_seed(T)
    codes = torch.tensor([0, 0x38, 0xB8, 0x40, 0xC0], dtype=torch.uint8, device="cuda")   # 0, 1, -1, 2, -2

    def rows(n):
        q = torch.empty((n, K), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // K)
        for i in range(0, n, step):
            part = q[i:i + step]
            part.copy_(codes[torch.randint(0, 5, part.shape, dtype=torch.int32, device="cuda", generator=gen)])
        s = torch.full((n, -(-K // 64), 2), 127, dtype=torch.uint8, device="cuda")
        if K % 64:
            s[:, -1, 1] = 0
        return q, s
    x, xs = rows(T)
    w, ws = rows(N)
    t, n = min(T, 200), min(N, 192 + N % 32)
    n0 = N - n
    assert n0 % 32 == 0   # whole blocks of the MXFP8 output
    res = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 1 << 14):
        part = res[i:i + (1 << 14)]
        part.copy_(torch.randint(-8, 9, part.shape, dtype=torch.int8, device="cuda", generator=gen))
    y = mx.mx_linear_fused(x, w, ws, x_s=xs, residual=res)
    part = mx.mx_linear_fused(x[-t:], w[n0:], ws[n0:], x_s=xs[-t:], residual=res[-t:, n0:].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(y[-t:, n0:], part)
    del res, y
    yq, ys = mx.mx_linear_fused(x, w, ws, x_s=xs, act="relu", quantize_out=True)
    pq, ps = mx.mx_linear_fused(x[-t:], w[n0:], ws[n0:], x_s=xs[-t:], act="relu", quantize_out=True)
    torch.cuda.synchronize()
    assert torch.equal(yq[-t:, n0:], pq) and torch.equal(ys[-t:].flatten(1)[:, n0 // 32:-(-N // 32)],
                                                       ps.flatten(1)[:, :-(-n // 32)])
