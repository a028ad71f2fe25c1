"""mx_linear_fused's tile kernels address the outputs of 8 rows by 32-bit byte
offsets: an output wide enough to pass them goes to the streaming kernels, whatever
its tokens."""

import random

import pytest

import mxfp8_block_scaled_topk_amd as mx

TILES = ("128x128", "256x128", "256x256")
EDGE = 1 << 27                         # the rule's
WRAPS = ((1 << 32) - 2 * 56) // 14     # past it, byte 2 (7 N + 56) of lane 63 no longer fits 32 bits


def most_tokens(N):   # fewer than 2^30 tiles of 32 x 32
    return 32 * (((1 << 30) - 1) // -(-N // 32))


@pytest.mark.parametrize("N", [EDGE, EDGE + 1, WRAPS, WRAPS + 1, 1 << 29, 1 << 30, (1 << 31) - 1])
def test_wide_outputs_take_no_tile_kernel(N):
    rng = random.Random(N)
    for T in [1, 33, 64, 65, 128, most_tokens(N)] + [rng.randint(1, most_tokens(N)) for _ in range(40)]:
        if T > most_tokens(N):
            continue
        for K in (32, 96, 512, 4096, 1 << 20):
            assert mx.linear_fused_kernel(T, K, N, True) not in TILES, (T, K)


def test_the_edge():
    """Below it they are taken, and their offsets fit."""
    assert EDGE - 1 < WRAPS and 2 * (7 * (EDGE - 1) + 56) < 1 << 32
    assert mx.linear_fused_kernel(128, 32, EDGE - 1, True) in TILES
