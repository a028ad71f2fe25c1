"""The INT8 operators and the expert sort run together, on one stream with no host
synchronisation, as they serve and as they train:

    q, s  = x quantised per token                    int8_quantize
    rows  = q and s sorted by expert                 moe_permute
    h     = silu(rows Wg^T) * (rows Wu^T)            gmm_int8 (SwiGLU)
    hq    = h quantised per row                      int8_quantize
    y     = hq Wd^T                                  gmm_int8
    m     = sum_j w y, back at the tokens            moe_unpermute
    out   = m Wo^T + bias + residual                 int8_linear

Every stage is checked on the GPU's own inputs of that stage; the chain is run
eagerly, captured, on two streams at once and with a padded batch.  The training
step's gradients are checked against float64 autograd."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from fused_util import F32_HALF, check_bf16
from gpu_util import bf16_dev, bf16_host, f32_dev, host, i32_dev, say
from oracle import int8_ref, mx_ref
from test_gpu_int8_products import reference, swiglu_bound
from test_gpu_permute import routes
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu


def weights(K, I, E, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def quantised(*shape):
        return mx.int8_quantize((torch.randn(shape, generator=gen, device="cuda") * 0.05).bfloat16())
    return dict(w13=quantised(E, 2 * I, K), w2=quantised(E, K, I), wo=quantised(K, K),
                bias=torch.randn(K, generator=gen, device="cuda"))


def layer(x, res, ids, w, d, E):
    """Everything the chain computes, in order."""
    q, s = mx.int8_quantize(x)
    rows = mx.moe_permute(q, ids, E, x_s=s)
    h = mx.gmm_int8(rows[0], rows[1], *d["w13"], rows[4], swiglu=True)
    hq = mx.int8_quantize(h)
    y = mx.gmm_int8(*hq, *d["w2"], rows[4])
    m = mx.moe_unpermute(y, rows[3], ids.shape[1], topk_w=w)
    out = mx.int8_linear(m, *d["wo"], bias=d["bias"], residual=res)
    return (q, s), rows, h, hq, y, m, out


def inputs(T, K, k, E, seed):
    rng = np.random.default_rng(seed)
    x = to_bf16_bits((rng.standard_normal((T, K)) * np.exp2(rng.integers(-2, 3, (T, 1)))).astype(np.float32))
    r = to_bf16_bits((2 * rng.standard_normal((T, K))).astype(np.float32))
    w = rng.random((T, k)).astype(np.float32)
    return x, r, routes(T, k, E, seed, skew=True), w / w.sum(axis=1, keepdims=True)


def check_layer(got, xb, rb, ids, w, d, E):
    (q, s), rows, h, hq, y, m, out = got
    T, k = ids.shape
    rq, rs = int8_ref.int8_quantize_ref(mx_ref.bf16_to_f64(xb))
    assert np.array_equal(host(q), rq) and np.array_equal(host(s), rs)
    px, sorted_row, eri, counts = int8_ref.permute_ref(rq, ids, E)
    n = sorted_row.size
    assert np.array_equal(host(rows[0])[:n], px) and np.array_equal(host(rows[1])[:n], rs[sorted_row // k])
    assert np.array_equal(host(rows[3]), eri) and np.array_equal(host(rows[4]), counts)
    ref, gu = int8_ref.gmm_int8_ref(px, rs[sorted_row // k], host(d["w13"][0]), host(d["w13"][1]), counts, True)
    check_bf16(mx_ref.bf16_to_f64(bf16_host(h)[:n]), ref, 0.0, swiglu_bound(ref, gu), "h")
    rq, rs = int8_ref.int8_quantize_ref(mx_ref.bf16_to_f64(bf16_host(h)[:n]))
    assert np.array_equal(host(hq[0])[:n], rq) and np.array_equal(host(hq[1])[:n], rs)
    ref, _ = int8_ref.gmm_int8_ref(rq, rs, host(d["w2"][0]), host(d["w2"][1]), counts, False)
    check_bf16(mx_ref.bf16_to_f64(bf16_host(y)[:n]), ref, 3.01 * F32_HALF, what="y")
    y64 = np.zeros((T * k, y.shape[1]))
    y64[:n] = mx_ref.bf16_to_f64(bf16_host(y)[:n])
    ref, mag = int8_ref.unpermute_ref(y64, eri, k, w), int8_ref.unpermute_ref(np.abs(y64), eri, k, w)
    check_bf16(mx_ref.bf16_to_f64(bf16_host(m)), ref, 0.0, 2 * k * F32_HALF * mag, "m")
    rq, rs = int8_ref.int8_quantize_ref(mx_ref.bf16_to_f64(bf16_host(m)))
    z = int8_ref.int8_product_ref(rq, rs, host(d["wo"][0]), host(d["wo"][1]))
    ref, err = reference(z, host(d["bias"]).astype(np.float64), "none", mx_ref.bf16_to_f64(rb))
    check_bf16(mx_ref.bf16_to_f64(bf16_host(out)), ref, 0.0, err, "out")


@pytest.mark.parametrize("T", [1, 33, 700])
def test_layer(T):
    K, I, E, k = 320, 112, 16, 4
    d = weights(K, I, E, T)
    xb, rb, ids, w = inputs(T, K, k, E, T)
    say(f"int8 layer T={T}")
    x, r, idd, wd = bf16_dev(xb), bf16_dev(rb), i32_dev(ids), f32_dev(w)
    got = layer(x, r, idd, wd, d, E)
    torch.cuda.synchronize()
    check_layer(got, xb, rb, ids, w, d, E)

    # captured: replays on new tokens and routes against the eager chain, eager work between
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer(x, r, idd, wd, d, E)[-1]
    for i in range(3):
        xb, rb, ids, w = inputs(T, K, k, E, 10 * T + i)
        for dst, src in ((x, bf16_dev(xb)), (r, bf16_dev(rb)), (idd, i32_dev(ids)), (wd, f32_dev(w))):
            dst.copy_(src)
        say(f"replay {i}")
        graph.replay()
        eager = layer(x.clone(), r.clone(), idd.clone(), wd.clone(), d, E)[-1]
        torch.cuda.synchronize()
        assert torch.equal(captured, eager), i


def test_padded_batch():
    """Tokens behind the batch have no experts; their rows of x are NaN and infinite."""
    T, real, K, I, E, k = 90, 61, 320, 112, 16, 4
    d = weights(K, I, E, 3)
    xb, rb, ids, w = inputs(T, K, k, E, 3)
    ids[real:] = -1
    x = bf16_dev(xb)
    x[real:] = float("nan")
    x[-1] = float("inf")
    got = layer(x, bf16_dev(rb), i32_dev(ids), f32_dev(w), d, E)
    clean = layer(bf16_dev(xb)[:real], bf16_dev(rb)[:real], i32_dev(ids[:real]), f32_dev(w[:real]), d, E)
    torch.cuda.synchronize()
    assert torch.equal(got[-1][:real], clean[-1])
    assert torch.equal(got[1][4], clean[1][4]) and not got[5][real:].any()


def test_two_streams_at_once():
    K, I, E, k, T = 512, 128, 16, 4, 300
    d = weights(K, I, E, 5)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [[inputs(T, K, k, E, 7 * i + j) for j in range(4)] for i in range(2)]
    on = [[(bf16_dev(x), bf16_dev(r), i32_dev(ids), f32_dev(w)) for x, r, ids, w in s] for s in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for j in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(*on[i][j], d, E)[-1])
    torch.cuda.synchronize()
    for i in range(2):
        for j in range(4):
            assert torch.equal(got[i][j], layer(*on[i][j], d, E)[-1]), (i, j)


def test_stream_argument():
    """Each entry point on a stream given by name, behind work that makes its inputs."""
    K, E, k, T = 512, 8, 2, 700
    side = torch.cuda.Stream()
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    new = torch.randn((T, K), device="cuda").bfloat16()
    ids = i32_dev(routes(T, k, E, 1))
    w8, ws = mx.int8_quantize(torch.randn((E, 64, K), device="cuda").bfloat16())
    w = torch.rand((T, k), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            x.copy_(new * 0)
        x.copy_(new)
    q, s = mx.int8_quantize(x, stream=side)
    rows = mx.moe_permute(q, ids, E, x_s=s, stream=side)
    y = mx.gmm_int8(rows[0], rows[1], w8, ws, rows[4], stream=side)
    out = mx.moe_unpermute(y, rows[3], k, topk_w=w, stream=side)
    dy, dw = mx.moe_unpermute_backward(out, rows[3], k, topk_w=w, y=y, stream=side)
    z = mx.int8_linear(x, w8[0], ws[0], stream=side)
    torch.cuda.synchronize()
    q2, s2 = mx.int8_quantize(new)
    rows2 = mx.moe_permute(q2, ids, E, x_s=s2)
    y2 = mx.gmm_int8(rows2[0], rows2[1], w8, ws, rows2[4])
    out2 = mx.moe_unpermute(y2, rows2[3], k, topk_w=w)
    dy2, dw2 = mx.moe_unpermute_backward(out2, rows2[3], k, topk_w=w, y=y2)
    z2 = mx.int8_linear(new, w8[0], ws[0])
    torch.cuda.synchronize()
    for a, b in ((q, q2), (s, s2), (rows[0], rows2[0]), (y, y2), (out, out2), (dy, dy2), (dw, dw2), (z, z2)):
        assert torch.equal(a, b)


def step(x, ids, w, We, dout, E):
    """Forward and backward of a routed layer of one matrix per expert, fp32 rows."""
    k = ids.shape[1]
    xp, _, _, eri, counts = mx.moe_permute(x, ids, E)
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), counts, output_size=xp.shape[0])
    y = torch.bmm(We[expert], xp[:, :, None])[:, :, 0]
    out = mx.moe_unpermute(y, eri, k, topk_w=w)
    dy, dw = mx.moe_unpermute_backward(dout, eri, k, topk_w=w, y=y)
    dxp = torch.bmm(We.transpose(1, 2).contiguous()[expert], dy[:, :, None])[:, :, 0]
    dWe = torch.zeros_like(We).index_add_(0, expert, dy[:, :, None] * xp[:, None, :])
    dx = mx.moe_unpermute(dxp, eri, k)
    return out, dx, dw, dWe


@pytest.mark.parametrize("T,K,N,E,k", [(1, 24, 9, 4, 2), (70, 33, 17, 6, 3), (300, 40, 64, 8, 2)])
def test_training_step(T, K, N, E, k):
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, dout = torch.randn((T, K), generator=gen, device="cuda"), torch.randn((T, N), generator=gen, device="cuda")
    We, w = torch.randn((E, N, K), generator=gen, device="cuda"), torch.rand((T, k), generator=gen, device="cuda")
    ids = i32_dev(routes(T, k, E, T))
    out, dx, dw, dWe = step(x, ids, w, We, dout, E)
    torch.cuda.synchronize()
    leaves = [t.double().cpu().requires_grad_() for t in (x, w, We)]
    chosen = leaves[2][ids.long().cpu()]                                  # [T, k, N, K]
    ref = torch.einsum("tk,tknc,tc->tn", leaves[1], chosen, leaves[0])
    ref.backward(dout.double().cpu())
    # sums of at most max(K, N) k products in fp32 at every step
    n = max(K, N) * k + T
    mags = [t.abs().double().cpu().requires_grad_() for t in (x, w, We)]
    mag = torch.einsum("tk,tknc,tc->tn", mags[1], mags[2][ids.long().cpu()], mags[0])
    mag.backward(dout.abs().double().cpu())
    for what, a, b, m in (("out", out, ref, mag), ("dx", dx, leaves[0].grad, mags[0].grad),
                          ("dw", dw, leaves[1].grad, mags[1].grad), ("dWe", dWe, leaves[2].grad, mags[2].grad)):
        assert ((a.double().cpu() - b).abs() <= (n + 4) * F32_HALF * m.detach()).all(), what


@pytest.mark.parametrize("dropped", [False, True])
def test_captured_backward(dropped):
    T, K, E, k = 260, 320, 16, 4
    ids = i32_dev(routes(T, k, E, 2))
    if dropped:
        ids[::7, 1] = -1   # (rows of dy that no entry names are zeros)
    x, w = torch.randn((T, K), device="cuda").bfloat16(), torch.rand((T, k), device="cuda")

    def run(x, w):
        xp, _, _, eri, _ = mx.moe_permute(x, ids, E)
        out = mx.moe_unpermute(xp, eri, k, topk_w=w)
        dy, dw = mx.moe_unpermute_backward(out, eri, k, topk_w=w, y=xp)
        return out, dy, dw, mx.moe_unpermute(dy, eri, k)
    run(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(x, w)
    for i in range(3):
        x.copy_(torch.randn((T, K), device="cuda"))
        w.copy_(torch.rand((T, k), device="cuda"))
        graph.replay()
        eager = run(x.clone(), w.clone())
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), i


def test_graphs_that_share_a_workspace():
    """Two captured sorts of different sizes and one of moe_route_quant, replayed in
    turn over one workspace."""
    E = 24
    shapes = [(300, 48, 8), (1100, 33, 3), (260, 64, 5)]
    need = max(mx.route_workspace_size(T, k, E) for T, _, k in shapes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    xs = [torch.randn((T, K), device="cuda").bfloat16() for T, K, _ in shapes]
    ids = [i32_dev(routes(T, k, E, T)) for T, _, k in shapes]

    def calls(i):
        if i == 2:
            return mx.moe_route_quant(xs[2], ids[2], E, workspace=ws)
        return mx.moe_permute(xs[i], ids[i], E, workspace=ws)
    graphs, got = [], []
    for i in range(3):
        calls(i)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            got.append(calls(i))
    for turn in range(4):
        for i in range(3):
            ids[i].copy_(i32_dev(routes(shapes[i][0], shapes[i][2], E, 10 * turn + i)))
            xs[i].copy_(torch.randn(xs[i].shape, device="cuda"))
            for t in got[i]:
                if t is not None:
                    t.zero_()
            say(f"turn {turn} graph {i}")
            graphs[i].replay()
            torch.cuda.synchronize()
            ref = int8_ref.permute_ref(host(xs[i].view(torch.int16)), host(ids[i]), E)
            maps = got[i][2:]
            for a, b in zip(maps, ref[1:]):
                assert np.array_equal(host(a), b), (turn, i)
            if i < 2:
                assert np.array_equal(host(got[i][0].view(torch.int16)), ref[0]), (turn, i)
