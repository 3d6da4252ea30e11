"""Pins of the oracle's norm, router and linear (CPU tier): closed forms,
brute force over all choices, and invariants."""
import itertools
import math

import numpy as np
import pytest

from oracle import bf16, linear, mxfp4, norm, router


def test_norm_closed_forms():
    h = np.array([[3.0, -4.0]])
    got = norm.rmsnorm(h, [1.0, 2.0], 2.0 ** -40)
    assert np.allclose(got, [[3 / math.sqrt(12.5), -8 / math.sqrt(12.5)]], rtol=1e-12)
    assert np.array_equal(norm.rmsnorm(np.zeros((2, 4)), np.ones(4), 1e-6), np.zeros((2, 4)))
    # eps alone: h far below it
    assert np.allclose(norm.rmsnorm(np.full((1, 4), 2.0 ** -60), np.ones(4), 0.25), 2.0 ** -59)


def test_residual_sum_rounds_once_to_its_type():
    x, r = 1.0, 2.0 ** -8                       # a tie of bfloat16: to even
    assert norm.residual_sum([x], [r], True)[0] == 1.0
    assert norm.residual_sum([x], [3 * r], True)[0] == 1.0 + 2.0 ** -6
    assert norm.residual_sum([x], [r], False)[0] == 1.0 + 2.0 ** -8
    assert bf16.decode(norm.round_y(np.array([1.0 + 2.0 ** -8 + 2.0 ** -40])))[0] == 1.0


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrtsoftplus"])
def test_scores_closed_forms(scoring):
    s = router.scores([0.0, math.log(3.0), -math.inf, math.nan], scoring)
    want = {"softmax": [0.25, 0.75], "sigmoid": [0.5, 0.75],
            "sqrtsoftplus": [math.sqrt(math.log(2.0)), math.sqrt(math.log(4.0))]}[scoring]
    assert np.allclose(s[:2], want, rtol=1e-14) and s[2] is None and s[3] is None


def test_router_against_all_choices():
    """Six experts, two of three groups, two experts: the chosen pair is the
    best among all pairs inside the best pair of groups."""
    rng = np.random.default_rng(3)
    for _ in range(50):
        l, b = rng.normal(size=6), 0.2 * rng.normal(size=6).astype(np.float32)
        ids, w = router.route_logits(l[None], 2, "sigmoid", b, 3, 2, True, 2.0)
        c = (1 / (1 + np.exp(-l))).astype(np.float32) + b
        rank = [c[2 * g] + c[2 * g + 1] for g in range(3)]
        groups = max(itertools.combinations(range(3), 2), key=lambda gs: sum(rank[g] for g in gs))
        pairs = itertools.combinations([e for g in groups for e in (2 * g, 2 * g + 1)], 2)
        best = max(pairs, key=lambda p: c[p[0]] + c[p[1]])
        assert set(ids[0]) == set(best) and c[ids[0, 0]] >= c[ids[0, 1]]
        assert abs(w.sum() - 2.0) < 1e-12


def test_router_ties_masks_and_empty_rows():
    inf = math.inf
    ids, w = router.route_logits([[1, 2, 2, 1], [-inf, 0, math.nan, -inf], [-inf] * 4, [inf, inf, 0, 0]], 3, "softmax",
                                 renormalize=False)
    assert ids.tolist() == [[1, 2, 0], [1, -1, -1], [-1, -1, -1], [0, 1, 2]]
    assert w[1].tolist() == [1, 0, 0] and w[2].tolist() == [0, 0, 0] and w[3].tolist() == [0.5, 0.5, 0]


@pytest.mark.parametrize("fp8", [False, True])
def test_linear_against_a_loop(fp8):
    rng = np.random.default_rng(5)
    x, wt = rng.normal(size=(3, 64)), rng.normal(size=(5, 64)).astype(np.float32)
    c, s = linear.quantize_tokens(bf16.decode(bf16.encode(x)), fp8)
    wc, ws = mxfp4.quantize_packed(wt)
    add = rng.normal(size=(3, 5))
    out, mag = linear.linear(c, s, wc, ws, fp8, add)
    from oracle import mxfp8
    xd, wd = (mxfp8 if fp8 else mxfp4).dequantize(c, s), mxfp4.dequantize(wc, ws)
    for t, n in itertools.product(range(3), range(5)):
        p = [xd[t, k] * wd[n, k] for k in range(64)]
        assert abs(out[t, n] - (math.fsum(p) + add[t, n])) < 1e-12
        assert abs(mag[t, n] - math.fsum(abs(v) for v in p)) < 1e-12
    assert np.all(linear.sum_error(mag, 64, fp8) < (2.0 ** -9 if fp8 else 2.0 ** -14) * mag)
