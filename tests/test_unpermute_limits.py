"""The most entries a token may have in moe_unpermute and its gradients: more are
refused on the host, and that many come out right."""

import ctypes

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx

UNSUPPORTED = -2
MOST = 1 << 20


def at(i):
    return ctypes.c_void_p((i + 1) << 40)   # never dereferenced


@pytest.mark.parametrize("K", [1, 64, 1 << 16])
@pytest.mark.parametrize("k", [MOST + 1, (1 << 31) - 8, (1 << 31) - 7, (1 << 31) - 2, (1 << 31) - 1])
def test_refused(k, K):
    """(up to 2^31 - 1, which T * k < 2^31 alone would let pass)"""
    lib = mx.load()
    for kind in (0, 1, 2):
        assert lib.moe_unpermute(at(0), kind, at(1), at(2), 1, K, k, 8, at(3), None) == UNSUPPORTED
        assert "2^20" in mx.last_error()
        assert lib.moe_unpermute_backward(at(0), kind, at(1), at(2), at(3), 1, K, k, 8, at(4), at(5), None) == UNSUPPORTED
        assert "2^20" in mx.last_error()


ROWS = [(torch.float32, 1), (torch.bfloat16, 3), (torch.float16, 40), (torch.bfloat16, 264), (torch.float32, 1000)]
CASES = [(T, k, dtype, K) for T, k in ((1, MOST), (3, MOST), (1, MOST - 1), (2, 99991)) for dtype, K in ROWS
         if T < 3 or K < 100]   # (the gradient's rows would take tens of GB)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,dtype,K", CASES)
def test_most_entries(T, k, dtype, K):
    """Small integers: every sum is exact."""
    gen = torch.Generator(device="cuda").manual_seed(k + K)
    draw = lambda hi, shape: torch.randint(-hi, hi + 1, shape, generator=gen, device="cuda")
    M = 1000
    y, w = draw(1, (M, K)).to(dtype), draw(1, (T, k)).float()
    eri = torch.randint(-M, M, (T * k,), generator=gen, device="cuda", dtype=torch.int32)   # half of them dropped
    eri[-1] = M - 1
    print(f"[gpu-case] moe_unpermute T={T} k={k} K={K} {dtype}", flush=True)
    out = mx.moe_unpermute(y, eri, k, topk_w=w)
    torch.cuda.synchronize()
    per_row = torch.zeros((T, M), dtype=torch.float64, device="cuda")   # the weights that each row gets
    kept = eri.view(T, k) >= 0
    for t in range(T):
        per_row[t].index_add_(0, eri.view(T, k)[t][kept[t]].long(), w[t][kept[t]].double())
    assert torch.equal(out, (per_row @ y.double()).to(dtype))   # (rounded once)

    rows = T * k
    place = torch.randperm(rows, generator=gen, device="cuda").int()
    place[::5] = -1
    d = draw(2, (T, K)).to(dtype)
    ys = draw(1, (rows, K)).to(dtype)
    dy = torch.full((rows, K), 7.0, dtype=dtype, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    print(f"[gpu-case] moe_unpermute_backward T={T} k={k} K={K} {dtype}", flush=True)
    mx.moe_unpermute_backward(d, place, k, topk_w=w, y=ys, out=(dy, dw))
    torch.cuda.synchronize()
    step = 1 << 16
    named = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for a in range(0, rows, step):
        p = place[a:a + step].long()
        i = torch.arange(a, min(a + step, rows), device="cuda")
        ok = p >= 0
        named[p[ok]] = True
        di = d[i // k].float()
        assert torch.equal(dy[p[ok]], (w.view(-1)[i][:, None] * di).to(dtype)[ok]), a
        want = (di * ys[p.clamp(min=0)].float()).sum(dim=1)
        assert torch.equal(dw.view(-1)[i], torch.where(ok, want, 0.0)), a
    assert (dy[~named] == 7).all()
