"""Residual addition and root-mean-square norm in fp64 (the definition in
include/moe_w4a4.h, moe_w4a4_add_rmsnorm)."""
from __future__ import annotations

import numpy as np

from . import bf16


def residual_sum(x, r, r_is_bf16: bool) -> np.ndarray:
    """x + r rounded once to the residual's type (bfloat16, or float32), as fp64 values.

    x is bfloat16 and r bfloat16 or float32, so the fp64 sum of two is within
    half a last bit of fp64 of exact; a residual in float32 is rounded to
    float32, one in bfloat16 to float32 first (the addition) and then to bfloat16.
    """
    s = (np.asarray(x, np.float64) + np.asarray(r, np.float64)).astype(np.float32).astype(np.float64)
    return bf16.decode(bf16.encode(s)) if r_is_bf16 else s


def rmsnorm(h, weight, eps: float) -> np.ndarray:
    """h * weight / sqrt(mean(h^2) + eps) along the last axis, unrounded."""
    h = np.asarray(h, np.float64)
    ms = np.mean(h * h, axis=-1, keepdims=True)
    return h * np.asarray(weight, np.float64) / np.sqrt(ms + float(np.float32(eps)))


def round_y(n) -> np.ndarray:
    """bf16 bits of n rounded to float32 first."""
    return bf16.encode(np.asarray(n, np.float64).astype(np.float32).astype(np.float64))
