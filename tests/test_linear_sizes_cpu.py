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


@pytest.mark.parametrize("T,K", [(1, 2048), (32, 2048), (1, 65536), (32, 32)])
def test_tokens_are_quantised_in_place_in_one_round_of_workgroups(T, K):
    """Few bf16 tokens need no workspace while the workgroups that each quantise
    them are no more than the 256 CUs, one per 32 features."""
    for N in (1, 96, 8191, 8192):
        assert mx.linear_fused_workspace_size(T, K, N, False) == 0
    for N in (8193, 16384, 131072):
        assert mx.linear_fused_workspace_size(T, K, N, False) >= T * K + T * 2 * -(-K // 64)
        assert mx.linear_fused_workspace_size(T, K, N, True) == 0


def test_which_kernel():
    """The query: the names' order, the bf16 tokens' kernel, refusals."""
    lib = mx.load()
    assert [mx.linear_fused_kernel(T, K, N, True) for T, K, N in
            ((1, 2048, 2048), (66, 256, 5650), (288, 640, 5400), (132, 256, 5493), (450, 256, 4104), (1030, 1664, 4096),
             (1440, 512, 5640))] == list(mx.LINEAR_KERNELS[:7])
    assert mx.linear_fused_kernel(32, 2048, 8192, False) == mx.LINEAR_KERNELS[7]
    assert mx.linear_fused_kernel(32, 2048, 8193, False) == mx.linear_fused_kernel(32, 2048, 8193, True)
    assert lib.mx_linear_fused_kernel(0, 64, 64, 1) == -1 and lib.mx_linear_fused_kernel(4, 0, 64, 1) == -1
    assert lib.mx_linear_fused_kernel(4, 65, 64, 1) == -2 and lib.mx_linear_fused_kernel(1 << 20, 32, 1 << 20, 1) == -2
    for sizes in ((0, 64, 64), (4, 65, 64)):
        with pytest.raises(mx.MxError):
            mx.linear_fused_kernel(*sizes, True)
