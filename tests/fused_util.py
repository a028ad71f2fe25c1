"""Comparison rules of the operators around the expert layer: an output that a
kernel computes in float32 and rounds once, against the float64 definition.

`rtol` and `atol` bound the kernel's float32 error before that rounding (each
test derives its own); the rounding adds half a step of the output's type.
"""

import numpy as np

from oracle.fused_ref import block_exponents
from oracle.mx_ref import e4m3_decode

BF16_HALF = 2.0 ** -8    # half of bf16's eps: a rounding's relative error
F32_HALF = 2.0 ** -24


def check_bf16(got, ref, rtol, atol=0.0, what=""):
    """got float64 values of a bf16 output, ref float64 before rounding."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = rtol * np.abs(ref) + atol
    tol = err + BF16_HALF * (np.abs(ref) + err) + 2.0 ** -134   # half a subnormal step
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])


def check_mx(q, s, ref, rtol, atol=0.0, what=""):
    """MXFP8 (q [R, K], s [R, ceil(K/64), 2] uint8) against float64 rows.

    A block's scale byte is the reference's, or that of the other side of a
    power of two which the block's maximum comes within its error of.  In the
    block's own scale a payload is off by its error plus half the e4m3 spacing
    at the code, or is the largest code with the reference at or beyond it.
    The byte that pads an odd count of scales is 0."""
    ref = np.asarray(ref, np.float64)
    R, K = ref.shape
    nb = -(-K // 32)
    assert q.shape == (R, K) and s.shape == (R, -(-K // 64), 2), what
    sb = s.reshape(R, -1).astype(np.int64)
    assert (sb[:, nb:] == 0).all(), (what, "padding byte")
    sb = sb[:, :nb]
    err = rtol * np.abs(ref) + atol
    lo, _ = block_exponents(np.maximum(np.abs(ref) - err, 0.0))
    hi, _ = block_exponents(np.abs(ref) + err)
    bad = (sb < lo + 127) | (sb > hi + 127)
    assert not bad.any(), (what, "scale", int(bad.sum()), np.argwhere(bad)[:4].tolist(), sb[bad][:4], lo[bad][:4])
    scale = np.repeat(np.exp2(sb - 127.0), 32, axis=1)[:, :K]
    code = q.astype(np.int64)
    deq = e4m3_decode(code) * scale
    ef = (code >> 3) & 0xF
    spacing = np.where(ef == 0, 2.0 ** -9, np.exp2(ef - 10.0)) * scale
    ok = np.abs(deq - ref) <= err + 0.5 * spacing * (1 + 1e-12)
    ok |= ((code & 0x7F) == 0x7E) & (np.sign(deq) * ref >= np.abs(deq) - err)
    assert ok.all(), (what, "payload", int((~ok).sum()), np.argwhere(~ok)[:4].tolist(), deq[~ok][:4], ref[~ok][:4])
