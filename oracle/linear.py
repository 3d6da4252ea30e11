"""The dense linear in fp64: out = Q(x) W^T (+ addend), and how far a
device's sums may be from it (the definition in include/moe_w4a4.h,
moe_w4a4_linear)."""
from __future__ import annotations

import numpy as np

from . import mxfp4, mxfp8


def quantize_tokens(x, fp8: bool):
    """(codes, scale bytes) of x as the layer's activations."""
    return (mxfp8 if fp8 else mxfp4).quantize_packed(x)


def linear(codes, scales, w_codes, w_scales, fp8: bool, addend=None):
    """(out fp64 [T, N], sum of the products' magnitudes [T, N])."""
    x = (mxfp8 if fp8 else mxfp4).dequantize(codes, scales)
    w = mxfp4.dequantize(w_codes, w_scales)
    out, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    return (out if addend is None else out + np.asarray(addend, np.float64)), mag


def sum_error(mag, K: int, fp8: bool):
    """Bound on a device's error before the output's rounding, from the
    magnitudes' sums `mag`.

    E2M1 products span 4 binades, so a matrix instruction's sum over one scale
    block is exact; aligning the blocks of a step and adding the accumulator
    loses less than 4 * 2^-21 of the largest term plus half a last bit (2^-24)
    of the sum, per step of 128, and the sum of up to 8 partial sums half a bit
    each: below (K/128 + 8) * 2^-18 of the magnitudes' sum at any order.
    E4M3 products are cut to multiples of 2^(ref - 13), 2^ref not above the
    largest product of eight neighbours: at most 8 * 2^-13 of it for the
    eight, so 2^-10 of the magnitudes' sum over all.
    """
    rel = (K // 128 + 9) * 2.0 ** -18 + (2.0 ** -10 if fp8 else 0.0)
    return rel * mag
