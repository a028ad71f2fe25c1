"""moe_route_mx and moe_mxfp8_forward_mx: bit-exact against the oracle's
permutation, and against the bf16 entry points on the rows those quantise."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import bf16_dev, guard_alloc, guards_intact, host, i32_dev, say, u8_dev
from oracle import fused_ref, moe_ref, mx_ref
from workloads import custom_config, make_inputs, to_bf16_bits

pytestmark = pytest.mark.gpu
NAMES = ("xq", "xs", "sorted_row", "expanded_row_idx", "group_list")


def draw(T, K, k, E, seed, skew=False):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, (T, K), dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] = 0x7E
    s = rng.integers(100, 140, (T, -(-K // 64), 2), dtype=np.uint8)
    if (K // 32) % 2:
        s[:, -1, 1] = 0
    p = np.arange(1, E + 1) ** -1.1 if skew else np.ones(E)
    ids = np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(T)]).astype(np.int32)
    return q, s, ids


@pytest.mark.parametrize("T,K,k,E", [
    (1, 32, 1, 1), (1, 2048, 8, 128), (3, 96, 2, 5), (32, 2048, 8, 128), (33, 64, 8, 8), (64, 4096, 4, 256),
    (300, 160, 3, 17), (257, 1024, 1, 40), (1031, 2048, 8, 64), (2049, 512, 6, 1024), (5, 65536, 2, 4),
])
def test_route_mx(T, K, k, E):
    q, s, ids = draw(T, K, k, E, T + K, skew=E > 16)
    M = T * k
    raws = [guard_alloc(M * K, torch.uint8), guard_alloc(M * (-(-K // 64)) * 2, torch.uint8),
            guard_alloc(M, torch.int32), guard_alloc(M, torch.int32), guard_alloc(E, torch.int64)]
    out = (raws[0][1].view(M, K), raws[1][1].view(M, -1, 2), raws[2][1], raws[3][1], raws[4][1])
    say(f"moe_route_mx T={T} K={K} k={k} E={E}")
    got = mx.moe_route_mx(u8_dev(q), u8_dev(s), i32_dev(ids), E, out=out)
    torch.cuda.synchronize()
    for name, g, r in zip(NAMES, got, fused_ref.route_mx_ref(q, s, ids, E)):
        assert np.array_equal(host(g), r), name
    for raw, t in raws:
        assert guards_intact(raw, t.numel() * t.element_size())


def test_route_mx_scale_alignment():
    """Scale tensors on odd addresses (copied byte by byte)."""
    T, K, k, E = 300, 512, 4, 16
    q, s, ids = draw(T, K, k, E, 1)
    sd = torch.empty(s.size + 1, dtype=torch.uint8, device="cuda")[1:].view(s.shape)
    sd.copy_(u8_dev(s))
    out = mx.moe_route_mx(u8_dev(q), sd, i32_dev(ids), E)
    torch.cuda.synchronize()
    for name, g, r in zip(NAMES, out, fused_ref.route_mx_ref(q, s, ids, E)):
        assert np.array_equal(host(g), r), name


def test_route_mx_dropped_assignments():
    """Ids outside [0, E) are dropped: their index is -1, and the rows behind the
    last expert's stay as they were."""
    T, K, k, E = 400, 128, 4, 8
    q, s, ids = draw(T, K, k, E, 2)
    flat = ids.reshape(-1)
    flat[::5] = -1
    flat[3::7] = E + 3
    M = T * k
    out = (torch.full((M, K), 0xA5, dtype=torch.uint8, device="cuda"),
           torch.full((M, K // 64, 2), 0xA5, dtype=torch.uint8, device="cuda"),
           torch.full((M,), -7, dtype=torch.int32, device="cuda"),
           torch.full((M,), -7, dtype=torch.int32, device="cuda"), torch.empty(E, dtype=torch.int64, device="cuda"))
    xq, xs, sr, eri, gl = (host(t) for t in mx.moe_route_mx(u8_dev(q), u8_dev(s), i32_dev(ids), E, out=out))
    valid = (flat >= 0) & (flat < E)
    order = np.nonzero(valid)[0][np.argsort(flat[valid], kind="stable")]
    n = order.size
    assert np.array_equal(gl, np.bincount(flat[valid], minlength=E))
    assert np.array_equal(sr[:n], order) and (sr[n:] == -7).all()
    assert (eri[~valid] == -1).all() and np.array_equal(eri[order], np.arange(n))
    assert np.array_equal(xq[:n], q[order // k]) and (xq[n:] == 0xA5).all()
    assert np.array_equal(xs[:n], s[order // k]) and (xs[n:] == 0xA5).all()


@pytest.mark.parametrize("limit", [0, 1])
def test_route_mx_bounded_wait(limit):
    """Workgroups that stop waiting for the counts count for themselves."""
    T, K, k, E = 1031, 256, 8, 64
    q, s, ids = draw(T, K, k, E, 3)
    old = mx.route_set_wait_limit(limit)
    try:
        out = mx.moe_route_mx(u8_dev(q), u8_dev(s), i32_dev(ids), E)
        torch.cuda.synchronize()
    finally:
        mx.route_set_wait_limit(old)
    for name, g, r in zip(NAMES, out, fused_ref.route_mx_ref(q, s, ids, E)):
        assert np.array_equal(host(g), r), name


def test_route_mx_equals_route_quant_of_quantised_rows():
    T, K, k, E = 2049, 2048, 8, 128
    rng = np.random.default_rng(4)
    x = bf16_dev(to_bf16_bits(rng.standard_normal((T, K)).astype(np.float32)))
    ids = i32_dev(draw(T, 32, k, E, 5)[2])
    q, s = mx.mx_quantize(x)
    for name, a, b in zip(NAMES, mx.moe_route_mx(q, s, ids, E), mx.moe_route_quant(x, ids, E)):
        assert torch.equal(a, b), name


def test_route_mx_empty():
    q, s, ids = (torch.empty((0, 64), dtype=torch.uint8, device="cuda"),
                 torch.empty((0, 1, 2), dtype=torch.uint8, device="cuda"),
                 torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    gl = mx.moe_route_mx(q, s, ids, 5)[4]
    torch.cuda.synchronize()
    assert host(gl).tolist() == [0] * 5


def test_route_mx_graph_replays_on_one_workspace():
    """Two captured graphs that share a workspace, replayed in turn on new ids,
    with eager calls on the same workspace between them."""
    T, K, k, E = 2049, 256, 8, 64
    sets = [draw(T, K, k, E, 30 + i, skew=i % 2 == 1) for i in range(4)]
    ws = torch.empty(mx.route_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    bufs = [tuple(t.clone() for t in (u8_dev(sets[0][0]), u8_dev(sets[0][1]), i32_dev(sets[0][2]))) for _ in range(2)]
    mx.moe_route_mx(*bufs[0], E, workspace=ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mx.moe_route_mx(*b, E, workspace=ws))
        graphs.append(g)
    for i in range(1, 4):
        for j in (0, 1):
            q, s, ids = sets[(i + j) % 4]
            for buf, new in zip(bufs[j], (u8_dev(q), u8_dev(s), i32_dev(ids))):
                buf.copy_(new)
            say(f"replay {i} of graph {j}")
            graphs[j].replay()
            torch.cuda.synchronize()
            ref = fused_ref.route_mx_ref(q, s, ids, E)
            for name, g, r in zip(NAMES, outs[j], ref):
                assert np.array_equal(host(g), r), (i, j, name)
            for name, g, r in zip(NAMES, mx.moe_route_mx(*bufs[j], E, workspace=ws), ref):
                assert np.array_equal(host(g), r), ("eager", i, j, name)


@pytest.mark.parametrize("fmt", [mx.WEIGHTS_E4M3, mx.WEIGHTS_E2M1, mx.WEIGHTS_PACKED])
@pytest.mark.parametrize("T", [1, 40, 600])
def test_forward_mx_equals_forward(fmt, T):
    """The layer on quantised rows gives the bytes of the layer that quantises
    the same rows itself."""
    cfg = custom_config("small", T, 512, 256, 16, 4)
    d = make_inputs(cfg)
    x, ids = bf16_dev(d["x"]), i32_dev(d["topk_ids"])
    w = torch.from_numpy(d["topk_w"]).cuda()
    w13, w2 = bf16_dev(d["w13"]), bf16_dev(d["w2"])
    if fmt == mx.WEIGHTS_E2M1:
        args = mx.mx_quantize_fp4(w13) + mx.mx_quantize_fp4(w2)
        ref = mx.moe_w4a8_forward(x, ids, w, *args)
    else:
        (a, a_s), (b, b_s) = mx.mx_quantize(w13), mx.mx_quantize(w2)
        args = (a, a_s, b, b_s)
        ref = mx.moe_mxfp8_forward(x, ids, w, *args)
        if fmt == mx.WEIGHTS_PACKED:
            args = (mx.mx_pack_weights(a, mx.PACK_GEMM1), a_s, mx.mx_pack_weights(b, mx.PACK_GEMM2), b_s)
    q, s = mx.mx_quantize(x)
    say(f"moe_mxfp8_forward_mx T={T} format={fmt}")
    got = mx.moe_mxfp8_forward_mx(q, s, ids, w, *args, weight_format=fmt)
    torch.cuda.synchronize()
    assert torch.equal(got, ref)
