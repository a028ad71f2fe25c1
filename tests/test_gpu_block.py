"""The operators around the expert layer run together, as half a transformer
block uses them, on one stream with no host synchronisation:

    h, n   = residual + x, its norm            mx_add_rmsnorm  (MXFP8 and bf16)
    ids, w = the router on bf16 n              moe_router
    m      = the experts on MXFP8 n            moe_mxfp8_forward_mx
    h, n   = h + m, its norm                   mx_add_rmsnorm  (MXFP8)
    f      = gelu(n W1^T + b1)                 mx_linear_fused (MXFP8 out)
    out    = f W2^T + b2 + h                   mx_linear_fused

Every stage is checked on the GPU's own inputs of that stage; the chain is run
eagerly, in place and captured, with the same bytes each way."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from fused_util import check_bf16, check_mx
from gpu_util import bf16_dev, bf16_host, bf16_rows_rel_err, check_router, f32_dev, host, say, u8_dev
from oracle import fused_ref, moe_ref, mx_ref
from test_gpu_linear_fused import reference
from test_gpu_norm import EPS, check as check_norm
from workloads import custom_config, make_inputs, router_inputs, to_bf16_bits

pytestmark = pytest.mark.gpu


def weights(K, I, E, F, seed):
    rng = np.random.default_rng(seed)
    d = make_inputs(custom_config("block", 4, K, I, E, 2), seed=seed)
    gate, _, _ = router_inputs(d["cfg"], d["x"])

    def quantised(n, k):
        w = to_bf16_bits((0.05 * rng.standard_normal((n, k))).astype(np.float32))
        return mx_ref.mx_quantize_ref(mx_ref.bf16_to_f64(w))
    w13, w2 = mx.mx_quantize(bf16_dev(d["w13"])), mx.mx_quantize(bf16_dev(d["w2"]))
    g = [(1 + 0.2 * rng.standard_normal(K)).astype(np.float32) for _ in range(2)]
    return dict(gate=gate, w13=w13, w2=w2, norm=g, up=quantised(F, K), down=quantised(K, F),
                b1=rng.standard_normal(F).astype(np.float32), b2=to_bf16_bits(rng.standard_normal(K).astype(np.float32)))


def on_device(wt):
    return dict(gate=bf16_dev(wt["gate"]), norm=[f32_dev(g) for g in wt["norm"]], w13=wt["w13"], w2=wt["w2"],
                up=[u8_dev(a) for a in wt["up"]], down=[u8_dev(a) for a in wt["down"]], b1=f32_dev(wt["b1"]),
                b2=bf16_dev(wt["b2"]))


def block(x, res, d, k, in_place=False):
    """Everything the chain computes, in order."""
    n1 = mx.mx_add_rmsnorm(x, d["norm"][0], res, EPS, norm_out=True,
                           out=None if not in_place else (*_mx_like(x), res, torch.empty_like(x)))
    ids, w = mx.moe_router(n1[3], d["gate"], k)
    m = mx.moe_mxfp8_forward_mx(n1[0], n1[1], ids, w, *d["w13"], *d["w2"])
    n2 = mx.mx_add_rmsnorm(m, d["norm"][1], n1[2], EPS, out=None if not in_place else (*_mx_like(x), n1[2], None))
    f = mx.mx_linear_fused(n2[0], *d["up"], x_s=n2[1], bias=d["b1"], act="gelu", quantize_out=True)
    y = mx.mx_linear_fused(f[0], *d["down"], x_s=f[1], bias=d["b2"], residual=n2[2],
                           out=n2[2] if in_place else None)
    return n1, ids, w, m, n2, f, y


def _mx_like(x):
    T, K = x.shape
    return (torch.empty((T, K), dtype=torch.uint8, device=x.device),
            torch.empty((T, -(-K // 64), 2), dtype=torch.uint8, device=x.device))


@pytest.mark.parametrize("T", [1, 33, 700])
def test_block(T):
    K, I, E, F, k = 512, 128, 16, 1120, 4
    wt = weights(K, I, E, F, T)
    d = on_device(wt)
    rng = np.random.default_rng(T + 1)
    xb = to_bf16_bits(rng.standard_normal((T, K)).astype(np.float32))
    rb = to_bf16_bits((2 * rng.standard_normal((T, K))).astype(np.float32))
    say(f"block T={T} K={K} I={I} E={E} F={F} k={k}")
    n1, ids, w, m, n2, f, y = block(bf16_dev(xb), bf16_dev(rb), d, k)
    torch.cuda.synchronize()

    check_norm(n1, xb, rb, wt["norm"][0].astype(np.float64), "first norm")
    yb = bf16_host(n1[3])
    check_router(host(ids), host(w), yb, wt["gate"], None, k, True)
    # the experts, on the norm's own rows
    q, s = host(n1[0]), host(n1[1])
    xq, xs, _, eri, counts = fused_ref.route_mx_ref(q, s, host(ids), E)
    hq, hs, _ = moe_ref.gmm_swiglu_mxquant_ref(xq, xs, host(d["w13"][0]), host(d["w13"][1]), counts, 1, I)
    ref = moe_ref.finalize_ref(moe_ref.gmm_mx_ref(hq, hs, host(d["w2"][0]), host(d["w2"][1]), counts, 1), host(w), eri)
    assert bf16_rows_rel_err(bf16_host(m), ref).max() <= 5e-2   # the layer's own end-to-end rule
    check_norm(n2, bf16_host(m), bf16_host(n1[2]), wt["norm"][1].astype(np.float64), "second norm")
    out, err = reference((host(n2[0]), host(n2[1])), wt["up"], wt["b1"].astype(np.float64), "gelu", None)
    check_mx(host(f[0]), host(f[1]), out, 0.0, err, "up")
    out, err = reference((host(f[0]), host(f[1])), wt["down"], mx_ref.bf16_to_f64(wt["b2"]), "none",
                         mx_ref.bf16_to_f64(bf16_host(n2[2])))
    check_bf16(mx_ref.bf16_to_f64(bf16_host(y)), out, 0.0, err, "down")

    # in place: the residual stream is one buffer throughout
    res = bf16_dev(rb)
    y2 = block(bf16_dev(xb), res, d, k, in_place=True)[-1]
    torch.cuda.synchronize()
    assert y2 is res and torch.equal(y2, y)

    # captured: replays on new tokens against the eager chain, eager work between
    x_buf, r_buf = bf16_dev(xb), bf16_dev(rb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = block(x_buf, r_buf, d, k)[-1]
    for i in range(3):
        nb = to_bf16_bits(rng.standard_normal((T, K)).astype(np.float32))
        x_buf.copy_(bf16_dev(nb))
        say(f"replay {i}")
        graph.replay()
        eager = block(bf16_dev(nb), bf16_dev(rb), d, k)[-1]
        torch.cuda.synchronize()
        assert torch.equal(captured, eager), i


def test_two_streams_at_once():
    """The chain on two streams at a time, each with its own buffers."""
    K, I, E, F, k, T = 512, 128, 16, 1120, 4, 300
    d = on_device(weights(K, I, E, F, 5))
    rng = np.random.default_rng(6)
    xs = [bf16_dev(to_bf16_bits(rng.standard_normal((T, K)).astype(np.float32))) for _ in range(2)]
    rs = [bf16_dev(to_bf16_bits(rng.standard_normal((T, K)).astype(np.float32))) for _ in range(2)]
    want = [block(x, r, d, k)[-1] for x, r in zip(xs, rs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for st, x, r in zip(streams, xs, rs):
            with torch.cuda.stream(st):
                got.append(block(x, r, d, k)[-1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [4, 40, 300, 700])
def test_rows_behind_a_batch(T):
    """Rows of NaN and infinities behind a batch (a padded one's unwritten
    rows) leave the other rows' bytes as they are, in every operator."""
    K, N, E, k, pad = 512, 640, 16, 4, 37
    rng = np.random.default_rng(T)
    xb = to_bf16_bits(rng.standard_normal((T + pad, K)).astype(np.float32))
    bad = xb.copy()
    bad[T:] = rng.choice(np.array([0x7FC0, 0x7F80, 0xFF80, 0x3F80], np.uint16), (pad, K))
    g = bf16_dev(to_bf16_bits(rng.standard_normal(K).astype(np.float32)))
    wq, ws = mx.mx_quantize(bf16_dev(to_bf16_bits((0.05 * rng.standard_normal((N, K))).astype(np.float32))))
    ids = u8_dev(rng.permuted(np.tile(np.arange(E), (T + pad, 1)), axis=1)[:, :k].copy()).int()
    ids_bad = ids.clone()
    ids_bad[T:] = -1   # no expert
    say(f"rows behind a batch T={T}")
    got = []
    for bits, i in ((xb, ids), (bad, ids_bad)):
        x = bf16_dev(bits)
        q, s, h, y = mx.mx_add_rmsnorm(x, g, x, norm_out=True)
        rows = [q, s, h, y, mx.mx_linear_fused(x, wq, ws, act="gelu", residual=x.repeat(1, 2)[:, :N].contiguous()),
                mx.mx_linear_fused(q, wq, ws, x_s=s, act="silu"),
                *mx.mx_linear_fused(q, wq, ws, x_s=s, quantize_out=True)]
        payload = q.clone()
        if bits is bad:
            payload[T:] = 0x7F   # NaN
        rows.append(mx.mx_linear_fused(payload, wq, ws, x_s=s))
        xq, xs, _, eri, _ = mx.moe_route_mx(q, s, i, E)
        at = eri[:T * k].long()
        torch.cuda.synchronize()
        assert int(at.min()) >= 0
        got.append([r[:T] for r in rows] + [xq[at], xs[at]])
    assert all(torch.equal(a, b) for a, b in zip(*got))
