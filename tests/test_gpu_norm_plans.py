"""mx_add_rmsnorm on batches of more rows than the GPU has CUs, where a row is
shared by fewer waves and holds more chunks a lane: every plan of its launch,
rows of 16-byte pieces and rows of any length.  Definition and bound are
test_gpu_norm's."""

import pytest
import torch

import mxfp8_block_scaled_topk_amd as mx
from gpu_util import bf16_dev, guard_alloc, guards_intact, say
from test_gpu_norm import EPS, check, make

pytestmark = pytest.mark.gpu

# waves a row x chunks a lane: 1 x 1, 1 x 2, 1 x 4, 4 x 2, 4 x 4, 8 x 4, 16 x 4 (aligned only), two passes
LENGTHS = [8, 509, 512, 520, 1000, 1021, 1024, 1032, 2041, 2048, 2056, 4093, 4096, 4104, 4304, 8190, 8192, 8200, 16383,
           16384, 16392, 32768]


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("residual,wf32", [(True, False), (True, True), (False, False)])
def test_norm_of_many_rows(K, residual, wf32):
    T = 301
    assert T > torch.cuda.get_device_properties(0).multi_processor_count
    x, r, w, w64 = make(T, K, residual, wf32, K)
    raws = [guard_alloc(T * K, torch.uint8), guard_alloc(T * -(-K // 64) * 2, torch.uint8),
            guard_alloc(T * K, torch.bfloat16), guard_alloc(T * K, torch.bfloat16)]
    out = (raws[0][1].view(T, K), raws[1][1].view(T, -1, 2), raws[2][1].view(T, K) if residual else None,
           raws[3][1].view(T, K))
    say(f"mx_add_rmsnorm T={T} K={K} residual={residual} fp32 weight={wf32}")
    got = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r) if residual else None, EPS, out=out)
    torch.cuda.synchronize()
    assert all(guards_intact(raw, t.numel() * t.element_size()) for raw, t in raws)
    check(got, x, r, w64, f"T={T} K={K}")


@pytest.mark.parametrize("K", LENGTHS)
def test_norm_of_many_rows_in_place_and_strided(K):
    """The residual stream and the rows in place; rows that are apart."""
    T = 301
    x, r, w, _ = make(T, K, True, True, K + 1)
    full = mx.mx_add_rmsnorm(bf16_dev(x), w, bf16_dev(r), EPS, norm_out=True)
    xd, rd = bf16_dev(x), bf16_dev(r)
    say(f"mx_add_rmsnorm T={T} K={K} in place")
    q, s = torch.empty_like(full[0]), torch.empty_like(full[1])
    mx.mx_add_rmsnorm(xd, w, rd, EPS, out=(q, s, rd, xd))
    for a, b in zip((q, s, rd, xd), full):
        assert torch.equal(a, b)
    wide = torch.zeros(T, K + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = bf16_dev(x)
    apart = mx.mx_add_rmsnorm(wide[:, :K], w, bf16_dev(r), EPS, norm_out=True)
    torch.cuda.synchronize()
    for a, b in zip(apart, full):
        assert torch.equal(a, b)


def test_norm_of_rows_over_several_rounds():
    """More rows than the grid has workgroups, in a plan of several chunks a lane."""
    T, K = 8197, 4304
    x, r, w, w64 = make(7, K, True, False, 1)
    xd, rd = (bf16_dev(t).repeat(T // 7, 1) for t in (x, r))
    say(f"mx_add_rmsnorm T={T} K={K}")
    got = mx.mx_add_rmsnorm(xd, w, rd, EPS, norm_out=True)
    torch.cuda.synchronize()
    check([t[:7] for t in got], x, r, w64, "rounds")
    for t in got:
        t = t.view(torch.uint8).view(T // 7, -1)
        assert bool((t == t[:1]).all())
