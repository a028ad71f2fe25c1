"""The oracle of the operators around the expert layer, pinned on the CPU:
closed forms, torch's own operations in float64, and the comparison rules
against planted mistakes."""

import numpy as np
import pytest
import torch

from fused_util import check_bf16, check_mx
from oracle import fused_ref, mx_ref


def test_rmsnorm_closed_forms():
    # a constant row normalises to its sign; a one-hot row of K elements to sqrt(K)
    w = np.ones(16)
    _, n = fused_ref.add_rmsnorm_ref(np.full((1, 16), -3.0), None, w, 1e-30)
    assert np.allclose(n, -1.0, rtol=1e-15)
    x = np.zeros((1, 16)); x[0, 5] = 7.0
    h, n = fused_ref.add_rmsnorm_ref(x, np.zeros((1, 16)), 2 * w, 1e-30)
    assert np.array_equal(h, x) and np.isclose(n[0, 5], 8.0) and np.count_nonzero(n) == 1


def test_rmsnorm_against_torch():
    rng = np.random.default_rng(0)
    x, r, w = rng.standard_normal((5, 33)), rng.standard_normal((5, 33)), rng.standard_normal(33)
    h, n = fused_ref.add_rmsnorm_ref(x, r, w, 1e-5)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x + r), (33,), torch.from_numpy(w), 1e-5).numpy()
    assert np.allclose(n, want, rtol=1e-13) and np.array_equal(h, x + r)


@pytest.mark.parametrize("act,fn", [
    ("none", lambda z: z), ("relu", torch.relu), ("silu", torch.nn.functional.silu),
    ("gelu", torch.nn.functional.gelu), ("gelu_tanh", lambda z: torch.nn.functional.gelu(z, approximate="tanh")),
])
def test_activations_against_torch(act, fn):
    z = np.concatenate([np.linspace(-12, 12, 4001), [-300.0, 300.0, 0.0]])
    got, want = fused_ref.activate_ref(z, act), fn(torch.from_numpy(z)).numpy()
    # torch's gelu computes 1 + erf, which keeps no more than 2^-53 |z| of the far tail
    assert np.all(np.abs(got - want) <= 1e-14 * np.abs(z) + 1e-13 * np.abs(want))


def test_linear_epilogue_order():
    x, w = np.array([[1.0, 2.0]]), np.array([[3.0, 4.0], [-5.0, 1.0]])
    got = fused_ref.linear_fused_ref(x, w, np.array([1.0, 1.0]), "relu", np.array([[10.0, 20.0]]))
    assert got.tolist() == [[22.0, 20.0]]     # relu(11 + 1) + 10, relu(-3 + 1) + 20


def test_route_mx_is_route_quant_of_the_same_rows():
    from oracle.moe_ref import route_quant_ref
    from workloads import to_bf16_bits
    rng = np.random.default_rng(1)
    x = to_bf16_bits(rng.standard_normal((9, 64)).astype(np.float32))
    ids = np.stack([rng.choice(6, 3, replace=False) for _ in range(9)]).astype(np.int32)
    q, s = mx_ref.mx_quantize_ref(mx_ref.bf16_to_f64(x))
    for a, b in zip(fused_ref.route_mx_ref(q, s, ids, 6), route_quant_ref(x, ids, 6)):
        assert np.array_equal(a, b)


def _quantised(K=70):
    rng = np.random.default_rng(2)
    v = rng.standard_normal((3, K)) * np.exp2(rng.integers(-9, 9, (3, 1)))
    return (v,) + mx_ref.mx_quantize_ref(v)


def test_check_mx_accepts_the_quantiser():
    v, q, s = _quantised()
    check_mx(q, s, v, 0.0)
    check_mx(q, s, v * (1 + 1e-7), 2e-7)


@pytest.mark.parametrize("plant", ["payload", "scale", "pad", "sign", "neighbour"])
def test_check_mx_rejects_mistakes(plant):
    v, q, s = _quantised()
    if plant == "payload":
        q[1, 3] += 2
    elif plant == "scale":
        s[0, 0, 1] += 1
    elif plant == "pad":
        s[2, 1, 1] = 7
    elif plant == "sign":
        q[0, 0] ^= 0x80
    else:
        q[2] = np.roll(q[2], 1)
    with pytest.raises(AssertionError):
        check_mx(q, s, v, 1e-6)


def test_check_bf16_counts_half_steps():
    ref = np.array([[1.0, 1.0]])
    check_bf16(np.array([[1.0 + 2.0 ** -8, 1.0 - 2.0 ** -9]]), ref, 0.0)
    with pytest.raises(AssertionError):
        check_bf16(np.array([[1.0 + 2.0 ** -7, 1.0]]), ref, 0.0)
