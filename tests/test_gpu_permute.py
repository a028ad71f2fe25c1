"""moe_permute bit for bit; moe_unpermute and its gradients against the float64
definition.

A token's sum takes k products and k - 1 additions in fp32, each off by half an
ulp of at most A = sum |w y|: 2 k 2^-24 A, then the rounding to the rows' type.
dw is a sum of K products in fp32, within (n + 1) 2^-24 of it in units of sum
|dout y|, n the additions that one product goes through: a lane's share of the
row, at most 8 for each 512 elements, then a tree over its lanes and waves."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import f32_dev, guard_alloc, guards_intact, host, i32_dev, say
from oracle import int8_ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}   # half a subnormal step
NAMES = ("xp", "sorted_row", "expanded_row_idx", "group_list")


def routes(T, k, E, seed, skew=False):
    rng = np.random.default_rng(seed)
    p = np.arange(1, E + 1) ** -1.1 if skew else np.ones(E)
    return np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(T)]).astype(np.int32)


def permute_out(T, K, k, E, dtype):
    raws = [guard_alloc(T * k * K, dtype), guard_alloc(T * k, torch.int32), guard_alloc(T * k, torch.int32),
            guard_alloc(E, torch.int64)]
    return raws, (raws[0][1].view(T * k, K), None, raws[1][1], raws[2][1], raws[3][1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "int8"])
@pytest.mark.parametrize("T,K,k,E", [
    (1, 1, 1, 1), (1, 2048, 8, 128), (3, 7, 2, 5), (3, 9, 2, 5), (32, 2048, 8, 128), (33, 17, 8, 8), (64, 1001, 4, 256),
    (300, 3, 3, 17), (257, 1024, 1, 40), (1031, 520, 8, 64), (2049, 133, 6, 1024), (5, 65537, 2, 4), (40, 20000, 8, 16),
    (300, 16, 2, 8), (600, 15, 4, 12),
])
def test_permute(T, K, k, E, dtype):
    dt = TYPES.get(dtype, torch.int8)
    gen = torch.Generator().manual_seed(T + K)
    x = torch.randint(-128, 128, (T, K * dt.itemsize), generator=gen, dtype=torch.int8).view(dt)   # any bytes at all
    ids = routes(T, k, E, T + K, skew=E > 16)
    raws, out = permute_out(T, K, k, E, dt)
    xs = sc = None
    if dtype == "int8":
        xs = torch.rand(T, generator=gen)
        sc = guard_alloc(T * k, torch.float32)
        raws.append(sc)
        out = (out[0], sc[1], *out[2:])
    say(f"moe_permute {dtype} T={T} K={K} k={k} E={E}")
    got = mx.moe_permute(x.cuda(), i32_dev(ids), E, x_s=None if xs is None else xs.cuda(), out=out)
    torch.cuda.synchronize()
    ref = int8_ref.permute_ref(x.view(torch.int8).numpy(), ids, E)
    assert np.array_equal(host(got[0].view(torch.int8)), ref[0])
    for name, g, r in zip(NAMES[1:], got[2:], ref[1:]):
        assert np.array_equal(host(g), r), name
    if xs is not None:
        assert np.array_equal(host(got[1]), xs.numpy()[ref[1] // k])
    for raw, t in raws:
        assert guards_intact(raw, t.numel() * t.element_size())


@pytest.mark.parametrize("T,K,k,E", [(30, 50, 2, 6), (700, 133, 4, 32)])
def test_permute_dropped_and_strided(T, K, k, E):
    """Ids outside [0, E) are dropped, the rows behind the last expert's stay; x's
    rows are strided and start on an odd element."""
    rng = np.random.default_rng(T)
    ids = routes(T, k, E, T)
    ids[rng.random((T, k)) < 0.2] = -1
    ids[rng.random((T, k)) < 0.1] = E
    ids[T - T // 8:] = np.iinfo(np.int32).min
    buf = torch.full((T * (K + 3) + 1,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = buf[1:].view(T, K + 3)[:, :K]
    x.copy_(torch.from_numpy(rng.standard_normal((T, K))).cuda())
    raws, out = permute_out(T, K, k, E, torch.bfloat16)
    got = mx.moe_permute(x, i32_dev(ids), E, out=out)
    torch.cuda.synchronize()
    rows, sorted_row, eri, counts = int8_ref.permute_ref(host(x.contiguous().view(torch.int16)), ids, E)
    n = int(counts.sum())
    assert np.array_equal(host(got[0].view(torch.int16))[:n], rows)
    assert np.array_equal(host(got[2])[:n], sorted_row) and np.array_equal(host(got[3]), eri)
    assert np.array_equal(host(got[4]), counts)
    fill = np.uint8(0xA5)
    assert (host(got[0][n:].contiguous().view(torch.uint8)) == fill).all() and (host(got[2][n:].view(torch.uint8)) == fill).all()
    for raw, t in raws:
        assert guards_intact(raw, t.numel() * t.element_size())


def test_permute_no_tokens_and_no_expert():
    x = torch.zeros((0, 64), dtype=torch.float16, device="cuda")
    got = mx.moe_permute(x, torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 9)
    torch.cuda.synchronize()
    assert got[0].shape == (0, 64) and not host(got[4]).any()
    got = mx.moe_permute(torch.ones((70, 64), device="cuda"), torch.full((70, 8), -1, dtype=torch.int32, device="cuda"), 9)
    torch.cuda.synchronize()
    assert not host(got[4]).any() and (host(got[3]) == -1).all()


def test_permute_past_32_bits():
    T, K, k, E = 140000, 8192, 2, 3      # 4.6 GB in, 9.2 GB out
    x = torch.zeros((T, K), dtype=torch.float32, device="cuda")
    x[:, 0] = torch.arange(T, device="cuda")
    x[:, -1] = -x[:, 0]
    ids = torch.stack([torch.arange(T, device="cuda") % 3, (torch.arange(T, device="cuda") + 1) % 3], dim=1).int()
    xp, _, sorted_row, eri, counts = mx.moe_permute(x, ids, E)
    token = (sorted_row // k).float()
    assert torch.equal(xp[:, 0], token) and torch.equal(xp[:, -1], -token) and not xp[:, 1:-1].any()
    back = mx.moe_unpermute(xp, eri, k)
    assert torch.equal(back, 2 * x)
    del back
    dy, _ = mx.moe_unpermute_backward(x, eri, k)
    assert torch.equal(dy, xp)


@pytest.mark.parametrize("polls", [0, 1])
def test_permute_wait_runs_out(polls):
    T, K, k, E = 1100, 96, 4, 20
    ids = routes(T, k, E, 3)
    x = torch.arange(T * K, dtype=torch.int32).view(T, K)
    before = mx.route_set_wait_limit(polls)
    try:
        got = mx.moe_permute(x.cuda(), i32_dev(ids), E)
        torch.cuda.synchronize()
    finally:
        mx.route_set_wait_limit(before)
    ref = int8_ref.permute_ref(x.numpy(), ids, E)
    assert np.array_equal(host(got[0]), ref[0]) and np.array_equal(host(got[3]), ref[2])


def dw_bound(K, mag):
    return (8 * -(-K // 512) + 16 + 1) * 2.0 ** -24 * mag + 1e-37


def rows_of(rng, shape, dtype):
    return torch.from_numpy((rng.standard_normal(shape) * np.exp2(rng.integers(-3, 3, (shape[0], 1)))).astype(np.float32)).to(TYPES[dtype])


def f64(t):
    return t.double().cpu().numpy()


def check(got, ref, err, dtype, what):
    got = f64(got)
    tol = err + HALF[dtype] * (np.abs(ref) + err) + TINY[dtype]
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])


SIZES = [   # T, K, k, more rows than T k
    (1, 1, 1, 0), (1, 2048, 8, 0), (3, 7, 2, 5), (5, 8, 3, 0), (33, 17, 8, 1), (64, 1001, 4, 0), (64, 4096, 2, 0),
    (257, 520, 1, 3), (300, 3, 3, 0), (100, 1024, 8, 0), (40, 2049, 9, 7), (9, 16384, 4, 0), (3, 40000, 2, 0), (2, 70001, 17, 0),
    (600, 256, 8, 0), (1, 5, 200, 0), (700, 2048, 4, 0), (5, 8200, 3, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_unpermute(i, dtype):
    T, K, k, more = SIZES[i]
    rng = np.random.default_rng(i)
    M = T * k + more
    y = rows_of(rng, (M, K), dtype)
    eri = rng.permutation(M)[:T * k].astype(np.int32)
    if i % 2:
        eri[rng.random(T * k) < 0.2] = rng.choice([-1, M, np.iinfo(np.int32).min, np.iinfo(np.int32).max])
        eri[:k] = -1   # a token with no row at all
        gone = np.setdiff1d(np.arange(M), eri)
        y[torch.from_numpy(gone)] = float("nan")   # rows that no entry names are not read
    w = rng.random((T, k)).astype(np.float32) if i % 3 else None
    raw, t = guard_alloc(T * K, TYPES[dtype])
    say(f"moe_unpermute {dtype} T={T} K={K} k={k} M={M} weighted={w is not None}")
    out = mx.moe_unpermute(y.cuda(), i32_dev(eri), k, topk_w=None if w is None else f32_dev(w), out=t.view(T, K))
    torch.cuda.synchronize()
    assert guards_intact(raw, T * K * TYPES[dtype].itemsize)
    y64 = np.nan_to_num(f64(y))
    ref = int8_ref.unpermute_ref(y64, eri, k, w)
    mag = int8_ref.unpermute_ref(np.abs(y64), eri, k, w)
    check(out, ref, 2 * k * 2.0 ** -24 * mag, dtype, "out")
    if i % 2:
        assert not f64(out)[0].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_unpermute_backward(i, dtype):
    T, K, k, more = SIZES[i]
    rng = np.random.default_rng(50 + i)
    M = T * k + more
    y, d = rows_of(rng, (M, K), dtype), rows_of(rng, (T, K), dtype)
    eri = rng.permutation(M)[:T * k].astype(np.int32)
    if i % 2:
        eri[rng.random(T * k) < 0.2] = rng.choice([-1, M])
        y[torch.from_numpy(np.setdiff1d(np.arange(M), eri))] = float("nan")
    w = rng.standard_normal((T, k)).astype(np.float32) if i % 3 else None
    want_dw = i % 4 != 3
    raws = [guard_alloc(M * K, TYPES[dtype]), guard_alloc(T * k, torch.float32)]
    say(f"moe_unpermute_backward {dtype} T={T} K={K} k={k} M={M} weighted={w is not None} dw={want_dw}")
    dy, dw = mx.moe_unpermute_backward(d.cuda(), i32_dev(eri), k, topk_w=None if w is None else f32_dev(w),
                                       y=y.cuda() if want_dw else None,
                                       out=(raws[0][1].view(M, K), raws[1][1].view(T, k) if want_dw else None))
    torch.cuda.synchronize()
    for raw, t in raws:
        assert guards_intact(raw, t.numel() * t.element_size())
    y64, d64 = np.nan_to_num(f64(y)), f64(d)
    ref, rw = int8_ref.unpermute_backward_ref(d64, eri, k, M, w, y64)
    named = ~np.isnan(ref[:, 0])
    check(dy[torch.from_numpy(named).cuda()], ref[named], 2.0 ** -24 * np.abs(ref[named]), dtype, "dy")
    left = dy[torch.from_numpy(~named).cuda()].contiguous().view(torch.uint8)
    assert (host(left) == 0xA5).all(), "rows that no entry names"
    if want_dw:
        mag = int8_ref.unpermute_backward_ref(np.abs(d64), eri, k, M, None, np.abs(y64))[1]
        assert (np.abs(host(dw) - rw) <= dw_bound(K, mag)).all()


def test_backward_without_out():
    """dy made by the call is zero in rows that no entry names; M = T k without y."""
    T, K, k = 6, 40, 3
    d = torch.randn((T, K), device="cuda")
    eri = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0)
    eri[4] = -1
    dy, dw = mx.moe_unpermute_backward(d, eri, k)
    torch.cuda.synchronize()
    assert dw is None and dy.shape == (T * k, K) and not dy[T * k - 5].any()
    kept = [i for i in range(T * k) if i != 4]
    assert torch.equal(dy[[T * k - 1 - i for i in kept]], d[[i // k for i in kept]])
    assert mx.moe_unpermute(d[:0], eri[:0], k).shape == (0, K)
    empty = mx.moe_unpermute_backward(d[:0], eri[:0], k, y=d)
    torch.cuda.synchronize()
    assert not empty[0].any() and empty[1].shape == (0, k)


def test_finalize_is_the_same():
    """moe_unpermute on bf16 rows gives moe_finalize's bits."""
    T, K, k = 500, 1024, 8
    y = torch.randn((T * k, K), device="cuda").bfloat16()
    w = torch.rand((T, k), device="cuda")
    eri = torch.randperm(T * k, device="cuda").int()
    eri[::17] = -1
    a, b = mx.moe_finalize(y, w, eri), mx.moe_unpermute(y, eri, k, topk_w=w)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("offset", [1, 3])
def test_odd_addresses(offset):
    """Every buffer on an odd element."""
    T, K, k = 37, 301, 4
    rng = np.random.default_rng(offset)
    M = T * k

    def shifted(t):
        buf = torch.zeros(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:].view(t.shape)
        return buf.copy_(t)
    for dtype in TYPES:
        y, d = rows_of(rng, (M, K), dtype), rows_of(rng, (T, K), dtype)
        eri, w = rng.permutation(M).astype(np.int32), rng.random((T, k)).astype(np.float32)
        yd, dd, ed, wd = shifted(y), shifted(d), shifted(torch.from_numpy(eri)), shifted(torch.from_numpy(w))
        out = mx.moe_unpermute(yd, ed, k, topk_w=wd, out=shifted(d))
        torch.cuda.synchronize()
        ref, mag = int8_ref.unpermute_ref(f64(y), eri, k, w), int8_ref.unpermute_ref(np.abs(f64(y)), eri, k, w)
        check(out, ref, 2 * k * 2.0 ** -24 * mag, dtype, "out")
        dy, dw = mx.moe_unpermute_backward(dd, ed, k, topk_w=wd, y=yd, out=(shifted(y), shifted(torch.from_numpy(w))))
        torch.cuda.synchronize()
        ref, rw = int8_ref.unpermute_backward_ref(f64(d), eri, k, M, w, f64(y))
        check(dy, ref, 2.0 ** -24 * np.abs(ref), dtype, "dy")
        mag = int8_ref.unpermute_backward_ref(np.abs(f64(d)), eri, k, M, None, np.abs(f64(y)))[1]
        assert (np.abs(host(dw) - rw) <= dw_bound(K, mag)).all()


def test_same_row_and_same_expert_twice():
    """A row that several entries name counts each time; ids that repeat within a
    token are assignments of their own."""
    T, K, k, M = 40, 264, 5, 7
    rng = np.random.default_rng(2)
    y, w = rows_of(rng, (M, K), "fp32"), rng.random((T, k)).astype(np.float32)
    eri = rng.integers(0, M, T * k).astype(np.int32)
    out = mx.moe_unpermute(y.cuda(), i32_dev(eri), k, topk_w=f32_dev(w))
    ref, mag = (int8_ref.unpermute_ref(v, eri, k, w) for v in (f64(y), np.abs(f64(y))))
    check(out, ref, 2 * k * 2.0 ** -24 * mag, "fp32", "out")
    # dw reads the shared rows (of dy they would be unspecified)
    d = rows_of(rng, (T, K), "fp32")
    _, dw = mx.moe_unpermute_backward(d.cuda(), i32_dev(eri), k, topk_w=f32_dev(w), y=y.cuda())
    mag = np.einsum("tc,tjc->tj", np.abs(f64(d)), np.abs(f64(y))[eri.reshape(T, k)])
    ref = np.einsum("tc,tjc->tj", f64(d), f64(y)[eri.reshape(T, k)])
    assert (np.abs(f64(dw) - ref) <= (K + 2) * 2.0 ** -24 * mag).all()
    for T in (9, 700):
        ids = np.repeat(rng.integers(0, 6, (T, 1)), 4, axis=1).astype(np.int32)
        x = rows_of(rng, (T, K), "fp32")
        got = mx.moe_permute(x.cuda(), i32_dev(ids), 6)
        torch.cuda.synchronize()
        ref = int8_ref.permute_ref(x.numpy(), ids, 6)
        assert np.array_equal(host(got[0]), ref[0])
        for a, b in zip(got[2:], ref[1:]):
            assert np.array_equal(host(a), b)


def test_differences():
    """The gradients against central differences of the operators themselves, in
    fp32 with steps and values that are exact: the loss is linear in each."""
    T, K, k, E = 12, 20, 3, 4
    rng = np.random.default_rng(8)
    ids = i32_dev(routes(T, k, E, 8))
    small = lambda *s: torch.from_numpy(rng.integers(-8, 9, s).astype(np.float32)).cuda()   # sums of exact integers
    x, w, d = small(T, K), small(T, k), small(T, K)
    _, _, sr, eri, _ = mx.moe_permute(x, ids, E)

    def loss(x, w):
        xp = mx.moe_permute(x, ids, E)[0]
        return float((mx.moe_unpermute(xp, eri, k, topk_w=w) * d).double().sum())
    xp = mx.moe_permute(x, ids, E)[0]
    dxp, dw = mx.moe_unpermute_backward(d, eri, k, topk_w=w, y=xp)
    dx = mx.moe_unpermute(dxp, eri, k)
    for grad, at_ in ((dx, 0), (dw, 1)):
        for _ in range(25):
            args = [x.clone(), w.clone()]
            i = tuple(int(rng.integers(n)) for n in grad.shape)
            args[at_][i] += 1
            up = loss(*args)
            args[at_][i] -= 2
            assert (up - loss(*args)) / 2 == float(grad[i])
