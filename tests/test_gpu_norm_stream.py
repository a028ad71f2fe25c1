"""mx_add_rmsnorm of strided leading dims with a stream of its own: the copies
that make rows of them belong to that stream, and there is one of each."""

import torch
import pytest

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import say

pytestmark = pytest.mark.gpu


def allocations():
    return torch.cuda.memory_stats()["allocation.all.allocated"]


@pytest.mark.parametrize("own_stream", [False, True])
def test_norm_copies_strided_rows_once(own_stream):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(6, 5, 96, device="cuda", generator=gen).bfloat16().transpose(0, 1) for _ in range(2))
    w = torch.ones(96, device="cuda")
    want = mx.mx_add_rmsnorm(x.contiguous(), w, r.contiguous(), norm_out=True)
    out = tuple(torch.empty_like(t) for t in want)
    stream = torch.cuda.Stream() if own_stream else None
    torch.cuda.synchronize()
    before = allocations()
    say(f"mx_add_rmsnorm of strided leading dims, own stream {own_stream}")
    mx.mx_add_rmsnorm(x, w, r, out=out, stream=stream)
    made = allocations() - before
    torch.cuda.synchronize()
    assert made == 2, made   # x's rows and the residual's
    assert all(torch.equal(a, b) for a, b in zip(out, want))
