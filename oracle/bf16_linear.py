"""The bfloat16 operators around the layer in fp64: linear, grouped linear,
experts, and the norm after a block (the definitions in include/moe_w4a4.h), and how
far a device's sums may be from them."""
from __future__ import annotations

import math

import numpy as np

from . import bf16, norm
from .route import route

FUNCTIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")     # by their MOE_FN_ numbers
# Largest slope of each (gelu's is 1.129 at sqrt 2, silu's 1.0998 near 2.4).
SLOPE = {"none": 1.0, "relu": 1.0, "silu": 1.11, "gelu": 1.13, "gelu_tanh": 1.13}


def apply(fn: str, v):
    v = np.asarray(v, np.float64)
    with np.errstate(over="ignore"):
        if fn == "relu":
            return np.where(v < 0, 0.0, v)
        if fn == "silu":
            return v / (1 + np.exp(-v))
        if fn == "gelu":
            return v * np.vectorize(lambda t: 0.5 * math.erfc(-t / math.sqrt(2)), otypes=[float])(v)
        if fn == "gelu_tanh":
            return v / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def linear(x, w, fn="none", gated=False, bias=None, row_scale=None, addend=None):
    """(out fp64 [T, N], bound [T, N] on a device's error before the output's rounding).

    A product of two bfloat16 values is exact in fp32.  A sum of K of them, in any order
    and with additions that may cut instead of round, is off by at most K * 2^-23 of
    the sum of the magnitudes, the partial sums' additions included; the bias adds half
    a last bit.  f passes an error on times its largest slope and is within 2^-20 of its
    value (and of fp32's smallest normal number); scale, product and addend round half
    a last bit each.
    """
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    K, half = x.shape[1], 2.0 ** -24
    v, err = x @ w.T, (K + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
        err = err + (np.abs(v) + err) * half
    n = v.shape[1] // 2 if gated else v.shape[1]
    out = apply(fn, v[:, :n])
    e = SLOPE[fn] * err[:, :n]
    if fn not in ("none", "relu"):
        e = e + np.abs(out) * 2.0 ** -20 + 2.0 ** -126
    if gated:
        up, eu = v[:, n:], err[:, n:]
        e = np.abs(up) * e + np.abs(out) * eu + e * eu
        out = out * up
        e = e + np.abs(out) * 2 * half
    if row_scale is not None:
        s = np.asarray(row_scale, np.float64)[:, None]
        out, e = out * s, e * np.abs(s)
        e = e + np.abs(out) * 2 * half
    if addend is not None:
        out = out + np.asarray(addend, np.float64)
        e = e + np.abs(out) * 2 * half
    return out, e + 2.0 ** -126


def grouped(x, w, offsets, rows=None, row_divisor=1, fn="none", gated=False, bias=None, row_scale=None, addend=None):
    """(out [R, N], bound) with NaN in the rows of no group; R rows of `rows` or x."""
    R = len(rows) if rows is not None else x.shape[0]
    n = w.shape[1] // 2 if gated else w.shape[1]
    out, err = np.full((R, n), np.nan), np.full((R, n), np.nan)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        at = np.arange(a, b) if rows is None else np.asarray(rows)[a:b] // row_divisor
        cut = lambda t: None if t is None else t[a:b]                                        # noqa: E731
        out[a:b], err[a:b] = linear(x[at], w[e], fn, gated, None if bias is None else bias[e], cut(row_scale), cut(addend))
    return out, err


def experts(x, ids, weights, w1, w2, fn="silu"):
    """The routed experts on bfloat16 values: out fp64 [T, H] from h and y rounded to bfloat16."""
    T, k = ids.shape
    _, offsets, order, pos = route(ids, w1.shape[0])
    if len(order) == 0:
        return np.zeros_like(x)
    h = bf16.decode(bf16.encode(grouped(x, w1, offsets, order, k, fn, True)[0]))
    y = bf16.decode(bf16.encode(grouped(h, w2, offsets)[0]))
    out = np.zeros((T, x.shape[1]))
    for r, p in enumerate(pos):
        if p >= 0:
            out[r // k] += float(weights[r // k, r % k]) * y[p]
    return out


def post_norm(x, residual, res_bf16, eps, post_weight=None, gate=None, scale=1.0):
    """(h unrounded, h rounded to the stream's type, bound on a device's error before that).
    A device's fp64 sums and products in another order are off by at most (cols + 12)
    roundings of 2^-53 of the step, and one of the sum."""
    z = np.asarray(x, np.float64)
    if post_weight is not None:
        z = norm.rmsnorm(z, post_weight, eps)
    step = z * float(np.float32(scale))
    if gate is not None:
        step = step * np.asarray(gate, np.float64)
    total = np.asarray(residual, np.float64) + step
    bound = (x.shape[1] + 12) * 2.0 ** -53 * np.abs(step) + 2.0 ** -52 * np.abs(total)
    return total, round_stream(total, res_bf16), bound


def round_stream(v, res_bf16: bool):
    """v rounded to float32, and a bfloat16 stream's to bfloat16 then."""
    v = np.asarray(v, np.float64).astype(np.float32).astype(np.float64)
    return bf16.decode(bf16.encode(v)) if res_bf16 else v
