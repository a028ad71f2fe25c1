"""int8_linear and gmm_int8 against the float64 definition.

The sum of products is exact.  Its conversion to fp32 and the two products with
the scales cost half an ulp each, 3 2^-24 |z| (the scales here keep z far from
fp32's ends), the bias another 2^-24 of the sum.  The activations' slopes stay
under 1.13, their own error is that of test_gpu_linear_fused.  SwiGLU: silu's
relative slope is at most 1 + |g|, so the gate's 3 2^-24 becomes (1 + |g|) 3 2^-24;
its exponential is within (|g| + 2) 2^-23, reciprocal and products within 2^-23
each: (2.5 |g| + 9) 2^-23 covers gate, up and products.  The reciprocal of 1 + e^-g
>= 2^126 is below the normal floats and comes out as 0: g <= -126 log 2 = -87.33, where
|silu(g)| = |g| / (1 + e^-g) is largest at that end, 87.34 2^-126 < 1.03e-36.  The
result is then off by less than 1.1e-36 |u|.
"""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from fused_util import F32_HALF, check_bf16
from gpu_util import bf16_dev, bf16_host, f32_dev, guard_alloc, guards_intact, host, i64_dev, say
from oracle import fused_ref, int8_ref, mx_ref
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def i8_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int8)).cuda()


def codes(rng, shape, spread=40.0):
    """int8 codes of a quantised normal, with the extremes among them."""
    q = np.clip(np.rint(rng.standard_normal(shape) * spread), -127, 127).astype(np.int8)
    flat = q.reshape(-1)
    flat[rng.integers(0, flat.size, max(1, flat.size // 50))] = -128
    return q


def scales(rng, shape, middle=0.01):
    return (middle * np.exp2(rng.uniform(-2, 2, shape))).astype(np.float32)


def reference(z, bias, act, res):
    """(out, its fp32 error bound), float64."""
    err = 3.01 * F32_HALF * np.abs(z)
    if bias is not None:
        z = z + bias
        err = err + F32_HALF * (np.abs(z) + err)
    a = fused_ref.activate_ref(z, act)
    err = 1.13 * err
    if act not in ("none", "relu"):
        err = err + (z * z + 4 * np.abs(z) + 16) * (1 + 0.1 * np.abs(z)) * 2.0 ** -23 * np.abs(a) + 1e-37
    out = a if res is None else a + res
    return out, err + F32_HALF * (np.abs(out) + err)


def linear_case(T, K, N, seed, int8_in=True, bias="none", act="none", residual=False, in_place=False, what=""):
    rng = np.random.default_rng(seed)
    wq, ws = codes(rng, (N, K)), scales(rng, N, 4 / (40 * 40 * np.sqrt(K)))
    if int8_in:
        xq, xs = codes(rng, (T, K)), scales(rng, T, 1.0)
        x, xsd = i8_dev(xq), f32_dev(xs)
    else:
        xb = to_bf16_bits((rng.standard_normal((T, K)) * np.exp2(rng.integers(-3, 3, (T, 1)))).astype(np.float32) * 40)
        xq, xs = int8_ref.int8_quantize_ref(mx_ref.bf16_to_f64(xb))
        x, xsd = bf16_dev(xb), None
    b = rng.standard_normal(N).astype(np.float32)
    bd, b64 = {"none": (None, None), "fp32": (f32_dev(b), b.astype(np.float64)),
               "bf16": (bf16_dev(to_bf16_bits(b)), mx_ref.bf16_to_f64(to_bf16_bits(b)))}[bias]
    rb = to_bf16_bits((2 * rng.standard_normal((T, N))).astype(np.float32)) if residual else None
    raw, t = guard_alloc(T * N, torch.bfloat16)
    out = t.view(T, N)
    res = None
    if residual:
        res = out.copy_(bf16_dev(rb)) if in_place else bf16_dev(rb)
    say(f"int8_linear {what} T={T} K={K} N={N} int8_in={int8_in} bias={bias} act={act} residual={residual} in_place={in_place}")
    y = mx.int8_linear(x, i8_dev(wq), f32_dev(ws), x_s=xsd, bias=bd, act=act, residual=res, out=out)
    torch.cuda.synchronize()
    assert guards_intact(raw, T * N * 2), what
    ref, err = reference(int8_ref.int8_product_ref(xq, xs, wq, ws), b64, act,
                         mx_ref.bf16_to_f64(rb) if residual else None)
    check_bf16(mx_ref.bf16_to_f64(bf16_host(y)), ref, 0.0, err, what)


SIZES = [
    (1, 16, 1), (1, 128, 64), (2, 48, 33), (1, 2048, 2048), (1, 4096, 512), (3, 80, 257), (8, 1024, 100), (9, 144, 31),
    (16, 2096, 255), (17, 384, 1000), (31, 4096, 96), (32, 240, 512), (32, 8192, 70), (33, 128, 64), (64, 256, 129),
    (65, 1024, 200), (127, 272, 65), (128, 2048, 256), (203, 2096, 515), (257, 400, 768), (300, 16, 300), (520, 4096, 192),
    (1100, 560, 1030), (2049, 256, 264), (513, 112, 517), (1, 131056, 3), (4, 65536, 40),
]


@pytest.mark.parametrize("i", range(len(SIZES)))
def test_linear(i):
    """Every size with two of the epilogues, all of which come up."""
    T, K, N = SIZES[i]
    for j in (0, 1):
        c = 2 * i + j
        linear_case(T, K, N, 100 + c, int8_in=c % 3 != 0, bias=["none", "bf16", "fp32"][(c + i) % 3], act=ACTS[c % 5],
                    residual=c % 4 < 2, in_place=c % 8 < 2, what=f"case {c}")


@pytest.mark.parametrize("T,K,N", [
    (1, 16, 5), (1, 2048, 4096), (1, 65536, 33), (2, 4112, 100), (3, 144, 257), (5, 2048, 8192), (7, 9360, 64), (13, 240, 70),
    (16, 4096, 96), (16, 16, 64), (15, 2064, 31), (9, 528, 8190), (1, 2048, 8224), (16, 4112, 40),
    (1, 16384, 33), (1, 16400, 33), (16, 1024, 8192), (16, 1040, 40), (2, 8192, 100), (3, 5456, 64), (15, 1088, 8191),
])
def test_few_bf16_tokens(T, K, N):
    """Tokens that every workgroup quantises itself, and the sizes just past them."""
    linear_case(T, K, N, T + K, int8_in=False, bias="fp32", act="silu", residual=True, what="bf16 tokens")
    if T <= 16 and T * K <= 16384 and N <= 8192:
        assert mx.int8_linear_workspace_size(T, K, N, False) == 0
    # the same codes and scales as int8_quantize's
    x = torch.randn((T, K), device="cuda").bfloat16()
    x[:, ::7] *= 30
    w, ws = i8_dev(codes(np.random.default_rng(1), (N, K))), torch.full((N,), 2.0 ** -10, device="cuda")
    q, s = mx.int8_quantize(x)
    a, b = mx.int8_linear(x, w, ws), mx.int8_linear(q, w, ws, x_s=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_extremes_are_exact():
    """Sums of the largest magnitude: +-128 * 128 * K, and cancelling ones."""
    K = 131056
    x = np.full((3, K), -128, np.int8)
    x[1, ::2] = 127
    x[2, :] = 127
    w = np.full((4, K), -128, np.int8)
    w[1, :] = 127
    w[2, ::2] = 1
    w[3, :] = 0
    w[3, K - 1] = 1
    xs, ws = np.float32([1, 0.5, 2]), np.float32([2.0 ** -20, 1, 2.0 ** -10, 3])
    y = mx.int8_linear(i8_dev(x), i8_dev(w), f32_dev(ws), x_s=f32_dev(xs))
    torch.cuda.synchronize()
    check_bf16(mx_ref.bf16_to_f64(bf16_host(y)), int8_ref.int8_product_ref(x, xs, w, ws), 3.01 * F32_HALF)


def test_rows_behind_the_batch_are_not_read():
    """NaN scales and extreme codes beyond T and N leave the results alone."""
    rng = np.random.default_rng(3)
    for T, K, N in ((5, 176, 70), (70, 240, 131), (300, 304, 515)):
        xq, wq = codes(rng, (T + 64, K)), codes(rng, (N + 64, K))
        xs, ws = scales(rng, T + 64, 0.01), scales(rng, N + 64, 0.01)
        xs[T:], ws[N:] = np.nan, np.nan
        b = rng.standard_normal(N + 64).astype(np.float32)
        b[N:] = np.nan
        y = mx.int8_linear(i8_dev(xq)[:T], i8_dev(wq)[:N], f32_dev(ws)[:N], x_s=f32_dev(xs)[:T], bias=f32_dev(b)[:N])
        torch.cuda.synchronize()
        ref, err = reference(int8_ref.int8_product_ref(xq[:T], xs[:T], wq[:N], ws[:N]), b[:N].astype(np.float64), "none", None)
        check_bf16(mx_ref.bf16_to_f64(bf16_host(y)), ref, 0.0, err, (T, K, N))


def swiglu_bound(y, gu):
    return (2.5 * np.abs(gu[0]) + 9) * 2.0 ** -23 * np.abs(y) + 1.1e-36 * np.abs(gu[1])


def experts_case(counts, K, N, swiglu, seed, kind=1, extra=0, what=""):
    """counts: rows per expert; `extra` rows behind them belong to nobody."""
    rng = np.random.default_rng(seed)
    E, M = len(counts), int(sum(counts)) + extra
    rows = 2 * N if swiglu else N
    aq, a_s = codes(rng, (M, K)), scales(rng, M, 1.0)
    wq, ws = codes(rng, (E, rows, K)), scales(rng, (E, rows), 3 / (40 * 40 * np.sqrt(K)))
    if extra:
        a_s[M - extra:] = np.nan
    gl = np.asarray(counts, np.int64)
    raw, t = guard_alloc(M * N, torch.bfloat16)
    out = t.view(M, N)
    before = bf16_host(out).copy()
    say(f"gmm_int8 {what} E={E} M={M} K={K} N={N} swiglu={swiglu} kind={kind} extra={extra}")
    y = mx.gmm_int8(i8_dev(aq), f32_dev(a_s), i8_dev(wq), f32_dev(ws), i64_dev(gl if kind == 1 else np.cumsum(gl)), kind,
                    swiglu=swiglu, out=out)
    torch.cuda.synchronize()
    assert guards_intact(raw, M * N * 2), what
    real = M - extra
    ref, g = int8_ref.gmm_int8_ref(aq[:real], a_s[:real], wq, ws, counts, swiglu)
    got = bf16_host(y)
    err = swiglu_bound(ref, g) if swiglu else 3.01 * F32_HALF * np.abs(ref)
    check_bf16(mx_ref.bf16_to_f64(got[:real]), ref, 0.0, err, what)
    assert np.array_equal(got[real:], before[real:]), (what, "rows that no expert owns")


EXPERTS = [
    ([1], 16, 1), ([0, 3, 0], 64, 33), ([2, 1, 0, 5, 2, 1, 1, 4], 2048, 96), ([1] * 40, 272, 65), ([33, 0, 32, 31], 144, 200),
    ([0, 0, 0, 70], 512, 128), ([64, 65, 63, 1], 400, 130), ([128, 127, 129], 256, 256), ([300, 2, 0, 257], 1024, 264),
    ([513, 1], 176, 515), ([17] * 60, 384, 48), ([1100, 0, 900], 240, 300), ([3] * 128, 256, 64), ([5, 250, 1, 0, 40] * 4, 640, 160),
]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("i", range(len(EXPERTS)))
def test_experts(i, swiglu):
    counts, K, N = EXPERTS[i]
    experts_case(counts, K, N, swiglu, 500 + i, kind=i % 2, extra=[0, 7, 40][i % 3], what=f"experts {i}")


def test_group_lists_are_clamped():
    """Lists that own more rows than there are, or negative counts, stay within the rows."""
    rng = np.random.default_rng(4)
    K, N, M = 128, 64, 50
    aq, a_s, wq, ws = codes(rng, (M, K)), scales(rng, M), codes(rng, (3, N, K)), scales(rng, (3, N))
    for gl, kind in (([20, 400, 9], 1), ([-5, 30, 30], 1), ([10, 5, 60], 0), ([1 << 40, 1, 1], 1), ([-(1 << 62), 1 << 62, 3], 1)):
        raw, t = guard_alloc(M * N, torch.bfloat16)
        y = mx.gmm_int8(i8_dev(aq), f32_dev(a_s), i8_dev(wq), f32_dev(ws), i64_dev(np.array(gl)), kind, out=t.view(M, N))
        torch.cuda.synchronize()
        assert guards_intact(raw, M * N * 2)
        counts = int8_ref.group_counts(gl, kind, M)
        n = int(counts.sum())
        ref, _ = int8_ref.gmm_int8_ref(aq[:n], a_s[:n], wq, ws, counts, False)
        check_bf16(mx_ref.bf16_to_f64(bf16_host(y)[:n]), ref, 3.01 * F32_HALF, what=str(gl))


def test_nobody_owns_a_row():
    out = torch.full((9, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    args = i8_dev(np.ones((9, 64))), f32_dev(np.ones(9)), i8_dev(np.ones((4, 32, 64))), f32_dev(np.ones((4, 32)))
    for kind in (0, 1):
        mx.gmm_int8(*args, i64_dev(np.zeros(4)), kind, out=out)
        torch.cuda.synchronize()
        assert (out == 5).all()
    assert mx.gmm_int8(args[0][:0], args[1][:0], args[2], args[3], i64_dev(np.zeros(4))).shape == (0, 32)
    assert mx.int8_linear(args[0][:0], args[2][0], args[3][0], x_s=args[1][:0]).shape == (0, 32)


def test_swiglu_saturates():
    """Gates far below and above zero: 0 and the product, no NaN."""
    K, N = 64, 32
    w = np.zeros((1, 2 * N, K), np.int8)
    w[0, :N, 0], w[0, N:, 1] = 127, 1
    a = np.zeros((4, K), np.int8)
    a[:, 0], a[:, 1] = [-127, 127, -1, 0], 3
    ws = np.ones((1, 2 * N), np.float32)
    y = mx.gmm_int8(i8_dev(a), f32_dev(np.ones(4)), i8_dev(w), f32_dev(ws), i64_dev([4]), swiglu=True)
    torch.cuda.synchronize()
    ref, g = int8_ref.gmm_int8_ref(a, np.ones(4, np.float32), w, ws, [4], True)
    check_bf16(mx_ref.bf16_to_f64(bf16_host(y)), ref, 0.0, swiglu_bound(ref, g))


def test_experts_as_the_linear():
    """One expert with every row is the dense product, bit for bit."""
    rng = np.random.default_rng(8)
    for T, K, N in ((40, 320, 100), (700, 256, 384)):
        xq, xs, wq, ws = codes(rng, (T, K)), scales(rng, T), codes(rng, (N, K)), scales(rng, N)
        a = mx.int8_linear(i8_dev(xq), i8_dev(wq), f32_dev(ws), x_s=f32_dev(xs))
        b = mx.gmm_int8(i8_dev(xq), f32_dev(xs), i8_dev(wq)[None], f32_dev(ws)[None], i64_dev([T]))
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_past_32_bits():
    """Weights, rows and outputs whose bytes lie past 4 GiB."""
    rng = np.random.default_rng(11)
    E, N, K = 40, 8192, 16384          # 5.4 GB of weights
    wq = torch.zeros((E, N, K), dtype=torch.int8, device="cuda")
    ws = torch.full((E, N), 2.0 ** -9, device="cuda")
    mine = codes(rng, (2, N, 64))
    wq[0, :, :64], wq[39, :, K - 64:] = i8_dev(mine[0]), i8_dev(mine[1])
    a = codes(rng, (6, K))
    counts = np.zeros(E, np.int64)
    counts[0], counts[39] = 2, 4
    y = mx.gmm_int8(i8_dev(a), f32_dev(np.ones(6)), wq, ws, i64_dev(counts))
    torch.cuda.synchronize()
    ref = np.concatenate([a[:2, :64].astype(np.float64) @ mine[0].T.astype(np.float64),
                          a[2:, K - 64:].astype(np.float64) @ mine[1].T.astype(np.float64)]) * 2.0 ** -9
    check_bf16(mx_ref.bf16_to_f64(bf16_host(y)), ref, 3.01 * F32_HALF)
    del wq, ws
    T, N, K = 300000, 8192, 16         # 4.9 GB out
    x = torch.zeros((T, K), dtype=torch.int8, device="cuda")
    pick = [0, 131071, 262143, 262144, T - 1]
    xq, w = codes(rng, (len(pick), K)), codes(rng, (N, K))
    x[pick] = i8_dev(xq)
    y = mx.int8_linear(x, i8_dev(w), f32_dev(np.ones(N)), x_s=torch.ones(T, device="cuda"))
    torch.cuda.synchronize()
    check_bf16(mx_ref.bf16_to_f64(bf16_host(y[pick])), xq.astype(np.float64) @ w.T.astype(np.float64), 3.01 * F32_HALF)
    assert int((y != 0).any(dim=1).sum()) == len(pick)
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("swiglu", [None, False, True])
def test_widest_outputs(swiglu):
    """N at its limit, where 16 rows of outputs span 4 GiB: each part equals a call on its weights."""
    T, K, N = 64, 16, (1 << 27) - 5
    gen = torch.Generator(device="cuda").manual_seed(1)

    def draw(*shape):
        return torch.randint(-128, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
    rows = 2 * N if swiglu else N
    x, xs, w, ws = draw(T, K), torch.rand(T, device="cuda"), draw(rows, K), torch.rand(rows, device="cuda") * 2.0 ** -12
    counts = i64_dev([T])
    res = torch.rand((T, N), device="cuda", dtype=torch.bfloat16) if swiglu is None else None
    say(f"N={N} swiglu={swiglu}")
    if swiglu is None:
        y = mx.int8_linear(x, w, ws, x_s=xs, residual=res)
    else:
        y = mx.gmm_int8(x, xs, w[None], ws[None], counts, swiglu=swiglu)
    step = 1 << 24
    for a in range(0, N, step):
        b = min(N, a + step)
        if swiglu is None:
            part = mx.int8_linear(x, w[a:b], ws[a:b], x_s=xs, residual=res[:, a:b].contiguous())
        elif swiglu:
            part = mx.gmm_int8(x, xs, torch.cat([w[a:b], w[N + a:N + b]])[None], torch.cat([ws[a:b], ws[N + a:N + b]])[None],
                               counts, swiglu=True)
        else:
            part = mx.gmm_int8(x, xs, w[a:b][None], ws[a:b][None], counts)
        assert torch.equal(y[:, a:b], part), a
    del x, w, ws, y, res, part
    torch.cuda.empty_cache()


def test_most_rows():
    """Row numbers up to 2^31 - 1, a tile's rounding past it."""
    M, K, N = (1 << 31) - 1, 16, 8
    rng = np.random.default_rng(5)
    pick = [0, (1 << 30) + 3, M - 1001, M - 1000, M - 2]
    mine, w = codes(rng, (len(pick), K)), codes(rng, (2, N, K))
    a = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    a[pick] = i8_dev(mine)
    a_s = torch.ones(M, device="cuda")
    for counts in ([M - 1000, 999], [0, M]):
        say(f"gmm_int8 M={M} counts={counts}")
        y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        mx.gmm_int8(a, a_s, i8_dev(w), torch.ones((2, N), device="cuda"), i64_dev(counts), out=y)
        torch.cuda.synchronize()
        e = [int(p >= counts[0]) for p in pick]
        ref = np.stack([w[j].astype(np.float64) @ m.astype(np.float64) for j, m in zip(e, mine)])
        check_bf16(mx_ref.bf16_to_f64(bf16_host(y[pick])), ref, 3.01 * F32_HALF)
        y[pick] = 0
        assert not y.any()
        del y
    del a, a_s
    torch.cuda.empty_cache()


def off(t, n=1):
    """The same values n elements past the start of an allocation."""
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
    view = buf[n:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("T,K,N", [(1, 144, 40), (5, 512, 77), (16, 1024, 512), (40, 272, 131), (203, 528, 515), (700, 256, 1030)])
def test_odd_addresses(T, K, N):
    """Everything but the int8 operands on any element: the outputs are the same."""
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda().bfloat16()
    w, ws = i8_dev(codes(rng, (N, K))), f32_dev(scales(rng, N))
    q, s = mx.int8_quantize(x)
    r = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).cuda().bfloat16()
    for b in (f32_dev(rng.standard_normal(N)), f32_dev(rng.standard_normal(N)).bfloat16()):
        for n in (1, 3):
            say(f"T={T} K={K} N={N} bias={b.dtype} offset={n}")
            a = mx.int8_linear(x, w, ws, bias=b, act="silu", residual=r)
            c = mx.int8_linear(off(x, n), w, off(ws, n), bias=off(b, n), act="silu", residual=off(r, n), out=off(r, n))
            d = off(r, n)
            d = mx.int8_linear(q, w, off(ws, n), x_s=off(s, n), bias=off(b, n), act="silu", residual=d, out=d)
            torch.cuda.synchronize()
            assert torch.equal(a, c) and torch.equal(a, d)
    for swiglu in (False, True):
        wr = w[:N // 2 * 2] if swiglu else w
        wsr = ws[:wr.shape[0]]
        counts = i64_dev([T // 2, T - T // 2])
        w2, ws2 = torch.stack([wr, wr.flip(0)]), torch.stack([wsr, wsr.flip(0)])
        a = mx.gmm_int8(q, s, w2, ws2, counts, swiglu=swiglu)
        c = mx.gmm_int8(q, off(s), w2, off(ws2), off(counts), swiglu=swiglu, out=off(torch.zeros_like(a)))
        torch.cuda.synchronize()
        assert torch.equal(a, c)
