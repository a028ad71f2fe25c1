"""The INT8 path's oracle against closed forms, brute force and differences."""

import numpy as np
import pytest

from oracle import int8_ref, mx_ref
from workloads import to_bf16_bits


def bf16(x):
    return mx_ref.bf16_to_f64(to_bf16_bits(np.asarray(x, np.float32)))


def test_quantiser_by_hand():
    q, s = int8_ref.int8_quantize_ref(np.array([[127.0, 1.0, -127.0, 0.5, 1.5, 2.5, -0.5, 0.0]]))
    assert s[0] == 1.0 and q.tolist() == [[127, 1, -127, 0, 2, 2, 0, 0]]   # ties to even
    q, s = int8_ref.int8_quantize_ref(np.zeros((2, 5)))
    assert not q.any() and (s == np.float32(2.0 ** -126)).all()
    q, s = int8_ref.int8_quantize_ref(np.full((1, 3), 2.0 ** -133))   # bf16's smallest
    assert s[0] == np.float32(2.0 ** -126) and not q.any()
    top = bf16([[3.3895e38, -3.3895e38, 1e30]])
    q, s = int8_ref.int8_quantize_ref(top)
    assert q.tolist() == [[127, -127, 0]] and np.isfinite(s).all()


def test_quantiser_of_no_number():
    q, s = int8_ref.int8_quantize_ref(np.array([[1.0, np.nan, np.inf], [1.0, -np.inf, 3e38], [1.0, -2.0, 0.0]]))
    assert np.isnan(s[0]) and s[1] == np.inf and not q[:2].any() and q[2].tolist() == [64, -127, 0]
    with np.errstate(invalid="ignore"):
        assert np.isnan(int8_ref.int8_product_ref(q[:2], s[:2], np.ones((4, 3)), np.ones(4))).all()


@pytest.mark.parametrize("scale", [1e-30, 1.0, 1e30])
def test_quantiser_error(scale):
    """A value is off by half a step, and 3 roundings of its 127 steps at most."""
    x = bf16(np.random.default_rng(3).standard_normal((50, 301)) * scale)
    q, s = int8_ref.int8_quantize_ref(x)
    assert (np.abs(q).max(axis=1) == 127).all()
    assert (np.abs(q * s.astype(np.float64)[:, None] - x) <= s[:, None] * (0.5 + 127 * 3 * 2.0 ** -24)).all()


def test_product_is_the_dequantised_one():
    rng = np.random.default_rng(0)
    a, b = rng.integers(-128, 128, (5, 48)).astype(np.int8), rng.integers(-128, 128, (7, 48)).astype(np.int8)
    sa, sb = rng.random(5).astype(np.float32), rng.random(7).astype(np.float32)
    z = int8_ref.int8_product_ref(a, sa, b, sb)
    for t in range(5):
        for n in range(7):
            total = sum(int(x) * int(y) for x, y in zip(a[t], b[n]))
            assert z[t, n] == total * float(sa[t]) * float(sb[n])


def test_group_counts():
    assert int8_ref.group_counts([2, 0, 3], 1, 10).tolist() == [2, 0, 3]
    assert int8_ref.group_counts([2, 2, 5], 0, 10).tolist() == [2, 0, 3]
    assert int8_ref.group_counts([2, 9, 5], 1, 6).tolist() == [2, 4, 0]
    assert int8_ref.group_counts([-3, 4, 5], 1, 6).tolist() == [0, 4, 2]


def test_permute_and_back():
    rng = np.random.default_rng(1)
    T, K, k, E = 40, 6, 3, 9
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int32)
    x = rng.standard_normal((T, K))
    rows, sorted_row, eri, counts = int8_ref.permute_ref(x, ids, E)
    flat = ids.reshape(-1)
    assert (np.diff(flat[sorted_row]) >= 0).all() and counts.tolist() == np.bincount(flat, minlength=E).tolist()
    assert np.array_equal(rows[eri], np.repeat(x, k, axis=0))
    assert np.allclose(int8_ref.unpermute_ref(rows, eri, k), k * x)
    assert np.allclose(int8_ref.unpermute_ref(rows, eri, k, np.full((T, k), 0.5)), 0.5 * k * x)


def test_gradients_against_differences():
    """The forward is linear in y and in w: differences over any step give the
    derivatives up to rounding."""
    rng = np.random.default_rng(2)
    T, K, k, M = 6, 5, 3, 20
    eri = rng.permutation(M)[:T * k].astype(np.int32)
    eri[[1, 7]] = -1
    w, y, dout = rng.random((T, k)), rng.standard_normal((M, K)), rng.standard_normal((T, K))
    dy, dw = int8_ref.unpermute_backward_ref(dout, eri, k, M, w, y)

    def loss(w, y):
        return (int8_ref.unpermute_ref(y, eri, k, w) * dout).sum()
    for t in range(T):
        for j in range(k):
            step = np.zeros((T, k))
            step[t, j] = 0.5
            assert np.isclose(loss(w + step, y) - loss(w - step, y), dw[t, j], atol=1e-12)
    for p in range(M):
        for c in range(K):
            step = np.zeros((M, K))
            step[p, c] = 0.5
            assert np.isclose(loss(w, y + step) - loss(w, y - step), np.nan_to_num(dy[p, c]), atol=1e-12)
    # the sort's own gradient is the way back without weights
    ids = np.stack([rng.choice(4, 2, replace=False) for _ in range(T)]).astype(np.int32)
    x, d = rng.standard_normal((T, K)), rng.standard_normal((2 * T, K))
    place = int8_ref.permute_ref(x, ids, 4)[2]
    dx = int8_ref.unpermute_ref(d, place, 2)
    for t in range(T):
        step = np.zeros((T, K))
        step[t, 1] = 0.5
        up, down = (int8_ref.permute_ref(x + sign * step, ids, 4)[0] for sign in (1, -1))
        assert np.isclose(((up - down) * d).sum(), dx[t, 1], atol=1e-12)
