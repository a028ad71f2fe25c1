"""mx_linear_fused's kernels one by one: the shapes name the kernel they are
for, and each test first asks linear_fused_kernel whether they still reach it.

Exact cases are small integers with power-of-two block scales: every product
and sum is exact in float32 in any order, so each output is the correctly
rounded one and is compared byte for byte at every position.  The others take
test_gpu_linear_fused's definition and bound on chosen rows."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from fused_util import check_bf16, check_mx
from gpu_util import bf16_dev, bf16_host, f32_dev, guard_alloc, guards_intact, host, say, u8_dev
from oracle import mx_ref
from test_gpu_linear_fused import ACTS, draw, reference
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu

# Tiles of several rounds: a workgroup's stage stream goes on into its next
# tile.  Even and odd numbers of k stages; scales a group of 4 stages at a time
# (K % 512 == 0), a stage at a time, and with an incomplete last stage.
ROUNDS = [
    ("256x256", 2691, 512, 8890), ("256x256", 5506, 1024, 4358), ("256x256", 2698, 1536, 8876),
    ("256x256", 2689, 640, 8833), ("256x256", 2837, 768, 8463), ("256x256", 3478, 544, 6921),
    ("256x256", 2819, 672, 8456),
    ("256x128", 2054, 1536, 7260), ("256x128", 1793, 1280, 8220), ("256x128", 1793, 1408, 8220),
    ("256x128", 2307, 1184, 6426), ("256x128", 2307, 1312, 6426),
    ("128x128", 1803, 512, 8267), ("128x128", 2049, 1024, 7197), ("128x128", 1033, 128, 7183),
    ("128x128", 1798, 256, 8205), ("128x128", 1793, 384, 8208), ("128x128", 1795, 160, 8219),
    ("128x128", 2050, 288, 7205), ("128x128", 907, 32, 8197),
]

# (kernel, shape with whole k stages, shape without): one round, incomplete last tiles
SHAPES = [
    ("32x32", (49, 256, 66), (65, 224, 75)),
    ("64x64", (66, 256, 5650), (65, 224, 5539)),
    ("64x96", (288, 640, 5400), (161, 1056, 5700)),
    ("64x64 twice per CU", (132, 256, 5493), (131, 224, 5472)),
    ("128x128", (450, 256, 4104), (449, 224, 4163)),
    ("256x128", (1030, 1664, 4096), (1030, 1696, 4099)),
    ("256x256", (1440, 512, 5640), (1443, 672, 5633)),
]
EACH = [pytest.param(name, *s, id=f"{name}-{'-'.join(map(str, s))}") for name, *two in SHAPES for s in two]


def reaches(name, T, K, N, x_is_mx=True):
    assert mx.linear_fused_kernel(T, K, N, x_is_mx) == name


def integers(T, K, N, seed):
    """e4m3 integers up to 15 and block scales near 1, and the float64 values."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rows(n, lo, hi):
        v = torch.randint(-15, 16, (n, K), device="cuda", generator=gen).float()
        nb = -(-K // 32)
        s = torch.zeros((n, -(-K // 64) * 2), dtype=torch.uint8, device="cuda")
        s[:, :nb] = torch.randint(lo, hi, (n, nb), device="cuda", generator=gen).byte()
        scale = torch.exp2(s[:, :nb].double() - 127).repeat_interleave(32, dim=1)[:, :K]
        return v.to(torch.float8_e4m3fn).view(torch.uint8), s.view(n, -1, 2), v.double() * scale
    (x, xs, x64), (w, ws, w64) = rows(T, 125, 129), rows(N, 126, 129)
    bias = torch.randint(-64, 65, (N,), device="cuda", generator=gen).float()
    res = torch.randint(-128, 129, (T, N), dtype=torch.int16, device="cuda", generator=gen).bfloat16()
    z = torch.mm(x64, w64.T.contiguous())
    assert float(z.abs().max()) < 2 ** 19   # 24 bits from the unit 2^-3
    return x, xs, w, ws, bias, res, z


def quantised(v):
    """MXFP8 bytes of exact float64 rows [R, N], by the format's definition."""
    R, N = v.shape
    nb = -(-N // 32)
    blocks = torch.nn.functional.pad(v, (0, nb * 32 - N)).view(R, nb, 32)
    top = blocks.abs().amax(dim=2)
    e = torch.where(top > 0, torch.frexp(top)[1].long() - 9, -127).clamp(-127, 127)
    t = (blocks * torch.exp2(-e.double())[:, :, None]).clamp(-448, 448).float()   # exact: a power of two
    q = t.to(torch.float8_e4m3fn).view(torch.uint8).view(R, -1)[:, :N].contiguous()
    s = torch.zeros((R, -(-N // 64) * 2), dtype=torch.uint8, device=v.device)
    s[:, :nb] = (e + 127).byte()
    return q, s.view(R, -1, 2)


def test_the_quantiser_of_the_exact_cases():
    v = np.random.default_rng(0).integers(-2000, 2000, (40, 100)).astype(np.float64) / 8
    for a, b in zip(quantised(torch.from_numpy(v).cuda()), mx_ref.mx_quantize_ref(v)):
        assert np.array_equal(host(a), b)


@pytest.mark.parametrize("name,T,K,N", ROUNDS)
def test_several_rounds_of_tiles(name, T, K, N):
    reaches(name, T, K, N)
    x, xs, w, ws, bias, res, z = integers(T, K, N, T + K)
    say(f"mx_linear_fused {name} T={T} K={K} N={N} rounds")
    raw, y = guard_alloc(T * N, torch.bfloat16)
    y = y.view(T, N)
    mx.mx_linear_fused(x, w, ws, x_s=xs, out=y)
    torch.cuda.synchronize()
    assert guards_intact(raw, 2 * T * N)
    assert torch.equal(y, z.float().bfloat16())

    raw, y = guard_alloc(T * N, torch.bfloat16)
    y = y.view(T, N)
    out = torch.relu(z + bias.double()) + res.double()
    mx.mx_linear_fused(x, w, ws, x_s=xs, bias=bias, act="relu", residual=res, out=y)
    torch.cuda.synchronize()
    assert guards_intact(raw, 2 * T * N)
    assert torch.equal(y, out.float().bfloat16())

    raws = [guard_alloc(T * N, torch.uint8), guard_alloc(T * -(-N // 64) * 2, torch.uint8)]
    q, s = raws[0][1].view(T, N), raws[1][1].view(T, -1, 2)
    mx.mx_linear_fused(x, w, ws, x_s=xs, bias=bias, act="relu", residual=res, out=(q, s))
    torch.cuda.synchronize()
    assert all(guards_intact(r, t.numel()) for r, t in raws)
    wq, wsc = quantised(out)
    assert torch.equal(q, wq) and torch.equal(s, wsc)


@pytest.mark.parametrize("name,T,K,N", EACH)
def test_exact_in_each_kernel(name, T, K, N):
    reaches(name, T, K, N)
    x, xs, w, ws, bias, res, z = integers(T, K, N, T + K)
    say(f"mx_linear_fused {name} T={T} K={K} N={N} exact")
    out = torch.relu(z + bias.double()) + res.double()
    y = mx.mx_linear_fused(x, w, ws, x_s=xs, bias=bias, act="relu", residual=res)
    q, s = mx.mx_linear_fused(x, w, ws, x_s=xs, bias=bias.bfloat16(), act="relu", residual=res, quantize_out=True)
    torch.cuda.synchronize()
    wq, wsc = quantised(out)
    assert torch.equal(y, out.float().bfloat16()) and torch.equal(q, wq) and torch.equal(s, wsc)


@pytest.mark.parametrize("name,T,K,N", EACH)
@pytest.mark.parametrize("act", ACTS)
def test_activations_in_each_kernel(name, T, K, N, act):
    """Each activation with bias and residual against the definition, on rows
    from every token fragment."""
    reaches(name, T, K, N)
    c = ACTS.index(act)
    xb, xq, wq = draw(T, K, N, 300 + c)
    rng = np.random.default_rng(c)
    b = rng.standard_normal(N).astype(np.float32)
    bd, b64 = [(None, None), (f32_dev(b), b.astype(np.float64)),
               (bf16_dev(to_bf16_bits(b)), mx_ref.bf16_to_f64(to_bf16_bits(b)))][(c + K // 32) % 3]
    rb = to_bf16_bits((2 * rng.standard_normal((T, N))).astype(np.float32)) if (c + K // 32) % 4 else None
    rows = np.unique(np.concatenate([np.arange(min(T, 3)), np.arange(max(0, T - 3), T), rng.integers(0, T, 20),
                                     np.arange(rng.integers(32), T, 32)]))
    res = None if rb is None else bf16_dev(rb)
    args = (u8_dev(xq[0]), u8_dev(wq[0]), u8_dev(wq[1]))
    say(f"mx_linear_fused {name} T={T} K={K} N={N} {act}")
    y = mx.mx_linear_fused(*args, x_s=u8_dev(xq[1]), bias=bd, act=act, residual=res)
    q, s = mx.mx_linear_fused(*args, x_s=u8_dev(xq[1]), bias=bd, act=act, residual=res, quantize_out=True)
    torch.cuda.synchronize()
    ref, err = reference((xq[0][rows], xq[1][rows]), wq, b64, act, None if rb is None else mx_ref.bf16_to_f64(rb[rows]))
    check_bf16(mx_ref.bf16_to_f64(bf16_host(y)[rows]), ref, 0.0, err, f"{name} {act}")
    check_mx(host(q)[rows], host(s)[rows], ref, 0.0, err, f"{name} {act}")


@pytest.mark.parametrize("name,T,K,N", EACH)
def test_placement_in_each_kernel(name, T, K, N):
    """The residual in place, buffers on odd addresses, and rolled batches give
    the bytes of the plain call."""
    reaches(name, T, K, N)
    xb, xq, wq = draw(T, K, N, 17)
    x, xs, w, ws = u8_dev(xq[0]), u8_dev(xq[1]), u8_dev(wq[0]), u8_dev(wq[1])
    res = bf16_dev(to_bf16_bits(np.random.default_rng(18).standard_normal((T, N)).astype(np.float32)))
    kw = dict(act="silu", bias=torch.linspace(-2, 2, N, device="cuda"))
    say(f"mx_linear_fused {name} T={T} K={K} N={N} placement")
    want = mx.mx_linear_fused(x, w, ws, x_s=xs, residual=res, **kw)
    wq8, ws8 = mx.mx_linear_fused(x, w, ws, x_s=xs, residual=res, quantize_out=True, **kw)
    r = res.clone()
    got = mx.mx_linear_fused(x, w, ws, x_s=xs, residual=r, out=r, **kw)
    torch.cuda.synchronize()
    assert got is r and torch.equal(r, want)

    def odd(t):
        o = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return o
    r = odd(res); r.copy_(res)
    b = odd(kw["bias"]); b.copy_(kw["bias"])
    y = mx.mx_linear_fused(x, w, ws, x_s=xs, residual=r, out=odd(want), act="silu", bias=b)
    q, s = mx.mx_linear_fused(x, w, ws, x_s=xs, residual=r, out=(odd(wq8), odd(ws8)), act="silu", bias=b)
    in_place = mx.mx_linear_fused(x, w, ws, x_s=xs, residual=r, out=r, act="silu", bias=b)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(q, wq8) and torch.equal(s, ws8) and torch.equal(in_place, want)

    shift = 77 % T
    rolled = mx.mx_linear_fused(x.roll(shift, 0), w, ws, x_s=xs.roll(shift, 0), residual=res.roll(shift, 0), **kw)
    torch.cuda.synchronize()
    assert torch.equal(rolled, want.roll(shift, 0))


@pytest.mark.parametrize("name,T,K,N", EACH)
def test_rows_behind_a_batch_in_each_kernel(name, T, K, N):
    """NaN payloads, NaN and infinite tokens and residuals in the last rows
    leave the others as they are; scales that say nothing but NaN too."""
    reaches(name, T, K, N)
    xb, xq, wq = draw(T, K, N, 19)
    keep = T - max(1, T // 3)
    x, xs, w, ws = u8_dev(xq[0]), u8_dev(xq[1]), u8_dev(wq[0]), u8_dev(wq[1])
    xf = bf16_dev(xb)
    res = torch.linspace(-3, 3, T * N, device="cuda").bfloat16().view(T, N)
    say(f"mx_linear_fused {name} T={T} K={K} N={N} rows behind")

    def run(x, xs, xf, res):
        return [t[:keep].clone() for t in (
            mx.mx_linear_fused(x, w, ws, x_s=xs, act="gelu", residual=res),
            *mx.mx_linear_fused(x, w, ws, x_s=xs, act="gelu_tanh", residual=res, quantize_out=True),
            mx.mx_linear_fused(xf, w, ws, act="silu"))]
    want = run(x, xs, xf, res)
    x, xs, xf, res = x.clone(), xs.clone(), xf.clone(), res.clone()
    x[keep:] = 0x7F
    xs[keep:] = 0xFF
    xf[keep:] = float("nan")
    xf[keep::2] = float("inf")
    res[keep:] = float("nan")
    got = run(x, xs, xf, res)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name,T,K,N", EACH)
def test_graphs_in_each_kernel(name, T, K, N):
    """Two graphs that share a workspace, replayed in turn on new tokens, each
    replay against the eager call, which runs between them."""
    reaches(name, T, K, N)
    assert mx.linear_fused_kernel(T, K, N, False) in (name, "32x32 bf16")
    gen = torch.Generator(device="cuda").manual_seed(T)
    w, ws = mx.mx_quantize((0.05 * torch.randn(N, K, device="cuda", generator=gen)).bfloat16())
    bufs = [torch.zeros(T, K, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    res = [torch.zeros(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    space = torch.empty(max(256, mx.linear_fused_workspace_size(T, K, N, False)), dtype=torch.uint8, device="cuda")
    kw = dict(act="gelu", bias=torch.linspace(-1, 1, N, device="cuda"))
    graphs, outs = [], []
    mx.mx_linear_fused(bufs[0], w, ws, residual=res[0], workspace=space, **kw)
    torch.cuda.synchronize()
    for b, r in zip(bufs, res):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((mx.mx_linear_fused(b, w, ws, residual=r, workspace=space, **kw),
                         *mx.mx_linear_fused(b, w, ws, residual=r, workspace=space, quantize_out=True, **kw)))
        graphs.append(g)
    for i in range(3):
        for j in (0, 1):
            bufs[j].copy_(torch.randn(T, K, device="cuda", generator=gen))
            res[j].copy_(torch.randn(T, N, device="cuda", generator=gen))
            say(f"{name} replay {i} of graph {j}")
            graphs[j].replay()
            eager = (mx.mx_linear_fused(bufs[j], w, ws, residual=res[j], **kw),
                     *mx.mx_linear_fused(bufs[j], w, ws, residual=res[j], quantize_out=True, **kw))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[j], eager)), (i, j)
