"""GPU tier: moe_w4a4_router against the fp64 oracle.

ids are whole numbers and have to be equal: what decides is a logit, or a score
computed in fp64 and rounded to float32, plus a float32 bias.  Weights are
float32 values with 32-bit statistics: with d = top - l an exponential is off by
at most (2 + d) * 2^-23 of itself, the softmax-weighted mean of d is at most
1 + ln(512) < 7.3, the sums of up to 512 terms, two quotients and the scale add
at most 13 roundings of 2^-24; 2^-18 relative covers all of it.  Scores below
2^-126 may lose their last bits: 2^-149 absolute, before a division by a sum
not below 1e-20."""
import math

import numpy as np
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from oracle import bf16, router
from tests.gpu_support import dev, dev_bf16, log

pytestmark = pytest.mark.gpu

SCORING = dict(softmax=_lib.MOE_SCORE_SOFTMAX, sigmoid=_lib.MOE_SCORE_SIGMOID, sqrtsoftplus=_lib.MOE_SCORE_SQRTSOFTPLUS)


def run(logits, k, scoring, bias=None, groups=1, keep=1, renorm=True, scale=1.0, half=False):
    T = logits.shape[0]
    l = dev_bf16(bf16_bits(logits)) if half else dev(logits.astype(np.float32))
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    _lib.moe_w4a4_router(l, ids[:T], w[:T], bias=None if bias is None else dev(bias), scoring=SCORING[scoring],
                         num_groups=groups, topk_groups=keep, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    assert torch.all(ids[T] == -7) and torch.all(w[T] == -7)           # rows behind the last
    return ids[:T].cpu().numpy(), w[:T].cpu().numpy().astype(np.float64)


def bf16_bits(v):
    fin = np.isfinite(v)
    out = bf16.encode(np.where(fin, v, 0.0))
    out[np.isposinf(v)], out[np.isneginf(v)], out[np.isnan(v)] = 0x7F80, 0xFF80, 0x7FC0
    return out


def check(logits, k, scoring, bias=None, groups=1, keep=1, renorm=True, scale=1.0, half=False):
    logits = bf16.decode(bf16_bits(logits)) if half else logits.astype(np.float32).astype(np.float64)
    ids, w = run(logits, k, scoring, bias, groups, keep, renorm, scale, half)
    rid, rw = router.route_logits(logits, k, scoring, bias, groups, keep, renorm, scale)
    assert np.array_equal(ids, rid), np.argwhere(ids != rid)[:4]
    tiny = 2.0 ** -149 * abs(scale) * (1e20 if renorm else 1.0)
    assert np.all(np.abs(w - rw) <= 2.0 ** -18 * np.abs(rw) + tiny), np.abs(w - rw).max()


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 2), (63, 5), (64, 6), (65, 16), (128, 8), (160, 6), (256, 6),
                                 (257, 1), (384, 8), (512, 16)])
@pytest.mark.parametrize("scoring", list(SCORING))
def test_sizes_and_scores(E, k, scoring):
    log(f"[test] router E {E} k {k} {scoring}")
    rng = np.random.default_rng(E + k)
    logits = 2 * rng.normal(size=(37, E))
    check(logits, k, scoring)
    check(logits, k, scoring, bias=(0.2 * rng.normal(size=E)).astype(np.float32), renorm=False, scale=2.5)
    check(logits, k, scoring, bias=(0.2 * rng.normal(size=E)).astype(np.float32), half=True)


@pytest.mark.parametrize("E,groups,keep,k", [(8, 8, 3, 3), (64, 8, 4, 6), (160, 8, 3, 8), (256, 8, 4, 8), (512, 64, 5, 16),
                                             (96, 3, 2, 4), (70, 7, 7, 6), (256, 2, 1, 8), (63, 63, 9, 9)])
@pytest.mark.parametrize("bias", [False, True])
def test_groups(E, groups, keep, k, bias):
    log(f"[test] router E {E} groups {groups} keep {keep} k {k} bias {bias}")
    rng = np.random.default_rng(groups)
    b = (0.3 * rng.normal(size=E)).astype(np.float32) if bias else None
    check(rng.normal(size=(41, E)), k, "sigmoid", b, groups, keep, scale=1.5)
    check(rng.normal(size=(41, E)), k, "softmax", b, groups, keep, half=True)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 1111, 4096])
def test_token_counts(T):
    log(f"[test] router T {T}")
    check(np.random.default_rng(T).normal(size=(T, 32)), 4, "sqrtsoftplus",
          np.linspace(-0.5, 0.5, 32, dtype=np.float32))


@pytest.mark.parametrize("scoring", list(SCORING))
def test_ties_go_to_the_lowest_index(scoring):
    log(f"[test] router ties {scoring}")
    rng = np.random.default_rng(1)
    logits = rng.integers(-2, 3, size=(60, 200)).astype(np.float64) / 2
    logits[0], logits[1] = 0.0, -0.0
    logits[2, ::2] = -0.0
    logits[2, 1::2] = 0.0
    check(logits, 12, scoring)
    check(logits, 12, scoring, bias=np.repeat(np.float32([0.25, 0.0]), 100))
    check(logits, 8, scoring, groups=20, keep=4)
    check(logits, 8, scoring, bias=np.zeros(200, np.float32), groups=20, keep=4, half=True)


@pytest.mark.parametrize("scoring", list(SCORING))
@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("bias", [False, True])
def test_masked_experts_and_rows(scoring, groups, keep, bias):
    """-infinity, NaN, the type's lowest value and +infinity in masked places;
    rows with fewer experts left than slots, with one, and with none."""
    log(f"[test] router masks {scoring} groups {groups} bias {bias}")
    rng = np.random.default_rng(2)
    inf = math.inf
    x = rng.normal(size=(14, 64))
    x[0] = -inf
    x[1] = math.nan
    x[2] = -inf
    x[2, 40] = 1.0
    x[3, 3:] = -inf
    x[4, ::2] = math.nan
    x[5] = np.finfo(np.float32).min
    x[6, 1:] = np.finfo(np.float32).min
    x[7, [9, 50]] = inf
    x[8] = inf
    x[9, 16:] = -inf
    x[10] = -800.0
    x[11] = 90.0 * rng.normal(size=64)
    x[12, :60] = -inf
    x[13, 5] = 1e30
    b = (0.1 * rng.normal(size=64)).astype(np.float32) if bias else None
    check(x, 6, scoring, b, groups, keep)
    check(x, 6, scoring, b, groups, keep, renorm=False)
    if bias:
        b[3], b[4], b[5] = -inf, math.nan, inf
        check(x, 6, scoring, b, groups, keep)


def test_near_equal_scores():
    """Scores a float32 step apart, and equal only after rounding."""
    log("[test] router near-equal scores")
    base = np.float32(0.731)
    steps = np.array([np.nextafter(base, np.float32(9)), base, np.nextafter(base, np.float32(-9))], np.float32)
    logits = np.tile(steps, (8, 30)).astype(np.float64)
    for s in SCORING:
        check(logits, 10, s, bias=np.zeros(90, np.float32))
        check(logits, 10, s)


def test_no_tokens():
    log("[test] router without tokens")
    _lib.moe_w4a4_router(torch.empty((0, 16), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                         torch.empty((0, 2), device="cuda"))
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last tokens against the oracle."""
    log("[test] router with offsets past 32 bits")
    T, E = 8_400_003, 257
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    tail = bf16.decode(bf16.encode(np.random.default_rng(4).normal(size=(21, E))))
    logits[-21:] = torch.from_numpy(tail).to(torch.bfloat16)
    ids = torch.empty((T, 5), dtype=torch.int32, device="cuda")
    w = torch.empty((T, 5), device="cuda")
    _lib.moe_w4a4_router(logits, ids, w)
    torch.cuda.synchronize()
    rid, rw = router.route_logits(tail, 5, "softmax")
    assert np.array_equal(ids[-21:].cpu().numpy(), rid)
    assert np.allclose(w[-21:].cpu().numpy(), rw, rtol=2.0 ** -18)
    assert torch.equal(ids[:-21], torch.arange(5, dtype=torch.int32, device="cuda").expand(T - 21, 5))


@pytest.mark.parametrize("scale", [0.0, -2.5])
def test_scale_of_any_sign(scale):
    log(f"[test] router scale {scale}")
    x = np.random.default_rng(5).normal(size=(7, 40))
    x[3, 2:] = -math.inf
    check(x, 4, "sigmoid", scale=scale)
    check(x, 4, "softmax", bias=np.zeros(40, np.float32), groups=5, keep=2, scale=scale, renorm=False)


def test_captured_and_replayed():
    log("[test] router captured")
    l, b = torch.randn((33, 160), device="cuda"), torch.randn(160, device="cuda") * 0.1
    ids, w = torch.empty((33, 8), dtype=torch.int32, device="cuda"), torch.empty((33, 8), device="cuda")
    call = lambda: _lib.moe_w4a4_router(l, ids, w, bias=b, scoring=SCORING["sqrtsoftplus"], num_groups=8,  # noqa: E731
                                        topk_groups=3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        l.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = ids.clone(), w.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], ids) and torch.equal(got[1], w)


def masked_top_rows(n, seed):
    """Rows whose largest logit is 70 above the rest and masked by the bias, so
    that every score in play is below 2^-90; the four experts left lie within
    2^-25 of a place half way between two float32 values of logit - 70 (2^-17
    apart), on either side of it."""
    rng = np.random.default_rng(seed)
    rows = np.empty((n, 6))
    rows[:, 0], rows[:, 1] = 70.0, -5.0
    place = rng.choice([-1, 1], size=(n, 1)) * (rng.integers(0, 512, size=(n, 1)) + 0.5) * 2.0 ** -17
    rows[:, 2:] = place + rng.integers(-32, 33, size=(n, 4)) * 2.0 ** -30
    return rows


def test_largest_logit_masked_by_the_bias():
    """The scores' differences then hang on the rounding of logit - largest."""
    log("[test] router, largest logit masked by the bias")
    ninf = -math.inf
    one = np.array([[70, float.fromhex("0x1.73bffep-8"), float.fromhex("0x1.73c002p-8"), -3]])
    check(one, 1, "softmax", np.array([ninf, 0, 0, 0], np.float32))
    two = np.array([[70, -5, 0.9967848062515259, 0.996761679649353, 0.9967756867408752, 0.9967743158340454]])
    check(two, 2, "softmax", np.array([ninf, ninf, 0, 0, 0, 0], np.float32), 3, 1)
    x = masked_top_rows(4000, 6)
    check(x, 1, "softmax", np.array([ninf, 0, 0, 0, 0, 0], np.float32))
    check(x, 3, "softmax", np.array([math.nan, 0, 0, 0, 0, 0], np.float32))
    check(x, 2, "softmax", np.array([ninf, ninf, 0, 0, 0, 0], np.float32), 3, 1)
    check(x, 2, "softmax", np.array([ninf, 0, 0, 0, 0, 0], np.float32), 3, 2)


def test_softmax_weights_far_below_the_largest_logit():
    """logit - largest at half a step of float32 between 64 and 87: the weights
    keep the bound of the nearer ones."""
    log("[test] router, softmax weights far below the largest")
    rng = np.random.default_rng(7)
    x = np.full((600, 4), -200.0)
    x[:, 0] = 70.0
    steps = rng.integers(0, 1 << 15, size=(600, 2)) * 2.0 ** -17
    x[:, 1:3] = rng.choice([-1, 1], size=(600, 2)) * (steps + 2.0 ** -18 - 2.0 ** -26)     # exact in float32
    check(x, 3, "softmax", renorm=False)
    check(x, 2, "softmax", np.array([-math.inf, 0, 0, 0], np.float32), renorm=False, scale=2.0 ** 60)
