"""mx_linear_fused refuses an output of 2^30 tiles or more on the host, before
its first launch (with bf16 tokens the quantiser comes first)."""

import ctypes

import pytest

import mxfp8_block_scaled_topk_amd as mx


def at(i):
    return ctypes.c_void_p((i + 1) << 44)   # 16 TiB apart, never dereferenced


@pytest.mark.parametrize("T,N", [((1 << 31) - 1, 513), (513, (1 << 31) - 1), (1 << 20, 1 << 20)])
def test_too_many_tiles(T, N):
    lib = mx.load()
    args = (at(0), None, at(1), at(2), None, 0, 0, None, T, 32, N, at(3), None, None, at(4), 1 << 43, None)
    assert lib.mx_linear_fused(*args) == -2 and "2^30" in mx.last_error()
    assert mx.linear_fused_workspace_size(T, 32, N, False) == 0
