"""moe_route_mx on rows of more than 128 MB, which it writes past the caches:
payloads, and scale rows of whole lines (K = 4096) or not."""

import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import guard_alloc, guards_intact, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,k,E", [(4160, 4096, 8, 64), (8256, 2048, 8, 128), (2700, 8192, 7, 60), (17000, 2080, 4, 33)])
def test_route_mx_past_the_caches(T, K, k, E):
    M = T * k
    assert M * K > 128 << 20
    gen = torch.Generator(device="cuda").manual_seed(T)
    q = torch.randint(0, 256, (T, K), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.randint(0, 256, (T, -(-K // 64), 2), dtype=torch.uint8, device="cuda", generator=gen)
    ids = torch.rand(T, E, device="cuda", generator=gen).argsort(dim=1)[:, :k].int().contiguous()
    raws = [guard_alloc(M * K, torch.uint8), guard_alloc(s.numel() * k, torch.uint8), guard_alloc(M, torch.int32),
            guard_alloc(M, torch.int32), guard_alloc(E, torch.int64)]
    out = (raws[0][1].view(M, K), raws[1][1].view(M, -1, 2), raws[2][1], raws[3][1], raws[4][1])
    flat = ids.view(-1).long()
    order = torch.argsort(flat, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(M, device="cuda")
    for i in range(2):
        say(f"moe_route_mx T={T} K={K} k={k} E={E} call {i}")
        xq, xs, sorted_row, eri, counts = mx.moe_route_mx(q, s, ids, E, out=out)
        torch.cuda.synchronize()
        assert all(guards_intact(raw, t.numel() * t.element_size()) for raw, t in raws)
        assert torch.equal(sorted_row.long(), order) and torch.equal(eri.long(), place)
        assert torch.equal(counts, torch.bincount(flat, minlength=E))
        assert torch.equal(xq, q[order // k]) and torch.equal(xs, s[order // k])
        for t in out:
            t.zero_()


def test_route_mx_past_the_caches_drops_assignments():
    """Ids outside [0, E): their rows are not written, nor any behind the last."""
    T, K, k, E = 8300, 4096, 8, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randint(0, 256, (T, K), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.randint(0, 256, (T, K // 64, 2), dtype=torch.uint8, device="cuda", generator=gen)
    ids = torch.rand(T, E, device="cuda", generator=gen).argsort(dim=1)[:, :k].int().contiguous()
    ids.view(-1)[::3] = -1
    ids.view(-1)[1::7] = E
    M = T * k
    out = (torch.full((M, K), 0xA5, dtype=torch.uint8, device="cuda"),
           torch.full((M, K // 64, 2), 0xA5, dtype=torch.uint8, device="cuda"),
           torch.full((M,), -7, dtype=torch.int32, device="cuda"),
           torch.full((M,), -7, dtype=torch.int32, device="cuda"), torch.zeros(E, dtype=torch.int64, device="cuda"))
    say(f"moe_route_mx T={T} K={K} k={k} E={E} dropped")
    xq, xs, sorted_row, eri, counts = mx.moe_route_mx(q, s, ids, E, out=out)
    torch.cuda.synchronize()
    flat = ids.view(-1).long()
    valid = (flat >= 0) & (flat < E)
    index = torch.nonzero(valid)[:, 0]
    order = index[torch.argsort(flat[index], stable=True)]
    n = order.numel()
    assert n * K > 128 << 20
    assert torch.equal(counts, torch.bincount(flat[index], minlength=E))
    assert torch.equal(sorted_row[:n].long(), order) and bool((sorted_row[n:] == -7).all())
    assert bool((eri[~valid] == -1).all()) and torch.equal(eri[order].long(), torch.arange(n, device="cuda"))
    assert torch.equal(xq[:n], q[order // k]) and bool((xq[n:] == 0xA5).all())
    assert torch.equal(xs[:n], s[order // k]) and bool((xs[n:] == 0xA5).all())


def test_forward_mx_past_the_caches():
    """The layer on such rows gives the bytes of the layer that quantises them itself."""
    T, K, I, E, k = 4160, 4096, 128, 32, 8
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, K, device="cuda", generator=gen).bfloat16()
    w, ids = torch.softmax(torch.randn(T, E, device="cuda", generator=gen), dim=1).topk(k)
    w13 = mx.mx_quantize((0.05 * torch.randn(E, 2 * I, K, device="cuda", generator=gen)).bfloat16())
    w2 = mx.mx_quantize((0.05 * torch.randn(E, K, I, device="cuda", generator=gen)).bfloat16())
    q, s = mx.mx_quantize(x)
    say(f"moe_mxfp8_forward_mx T={T} K={K}")
    got = mx.moe_mxfp8_forward_mx(q, s, ids.int(), w, *w13, *w2)
    want = mx.moe_mxfp8_forward(x, ids.int(), w, *w13, *w2)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
