"""Pins of the oracle's bfloat16 operators (CPU tier): closed forms, brute force and
invariants."""
import math

import numpy as np
import pytest
import torch

from oracle import bf16, bf16_linear


def test_functions_closed_forms():
    v = np.array([-30.0, -1.0, 0.0, 1.0, 30.0])
    assert np.array_equal(bf16_linear.apply("none", v), v)
    assert np.array_equal(bf16_linear.apply("relu", v), [0, 0, 0, 1, 30])
    for fn in ("silu", "gelu", "gelu_tanh"):
        f = bf16_linear.apply(fn, v)
        assert f[2] == 0 and abs(f[4] - 30) < 1e-10 and abs(f[0]) < 3e-12
        assert np.isclose(f[3] + -f[1], 1.0, rtol=1e-12) or fn == "none"          # f(v) - f(-v) = v
    assert np.isclose(bf16_linear.apply("silu", 1.0), 1 / (1 + math.exp(-1)), rtol=1e-15)
    assert np.isclose(bf16_linear.apply("gelu", 1.0), 0.8413447460685429, rtol=1e-14)
    assert np.isclose(bf16_linear.apply("gelu_tanh", 1.0), 0.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * 1.044715)), rtol=1e-14)


@pytest.mark.parametrize("fn", bf16_linear.FUNCTIONS)
def test_functions_against_torch_and_their_slopes(fn):
    v = np.linspace(-9, 9, 20001)
    t = torch.from_numpy(v)
    want = dict(none=t, relu=torch.relu(t), silu=torch.nn.functional.silu(t), gelu=torch.nn.functional.gelu(t),
                gelu_tanh=torch.nn.functional.gelu(t, approximate="tanh"))[fn].numpy()
    f = bf16_linear.apply(fn, v)
    assert np.allclose(f, want, rtol=1e-12, atol=1e-14)
    assert np.abs(np.diff(f) / np.diff(v)).max() <= bf16_linear.SLOPE[fn]


@pytest.mark.parametrize("gated", [False, True])
def test_linear_is_the_double_loop(gated):
    rng = np.random.default_rng(0)
    T, K, N = 3, 5, 4
    x, w = rng.normal(size=(T, K)), rng.normal(size=(2 * N if gated else N, K))
    b, s, a = rng.normal(size=w.shape[0]), rng.normal(size=T), rng.normal(size=(T, N))
    got, bound = bf16_linear.linear(x, w, "silu", gated, b, s, a)
    for t in range(T):
        for n in range(N):
            v = sum(x[t, k] * w[n, k] for k in range(K)) + b[n]
            f = v / (1 + math.exp(-v))
            if gated:
                f *= sum(x[t, k] * w[N + n, k] for k in range(K)) + b[N + n]
            assert math.isclose(got[t, n], a[t, n] + s[t] * f, rel_tol=1e-12)
    assert np.all(bound > 0)
    # a float32 evaluation stays within the bound
    f32 = lambda v: torch.from_numpy(np.asarray(v)).float()                          # noqa: E731
    x32, w32 = f32(bf16.decode(bf16.encode(x))), f32(bf16.decode(bf16.encode(w)))
    v = x32 @ w32.T + f32(b)
    f = torch.nn.functional.silu(v[:, :N]) * (v[:, N:] if gated else 1)
    out = f * f32(s)[:, None] + f32(a)
    ref, bound = bf16_linear.linear(x32.numpy(), w32.numpy(), "silu", gated, f32(b).numpy(), f32(s).numpy(), f32(a).numpy())
    assert np.all(np.abs(out.numpy() - ref) <= bound + np.abs(ref) * 2.0 ** -24)


def test_grouped_is_one_linear_a_group():
    rng = np.random.default_rng(1)
    x, w = rng.normal(size=(4, 8)), rng.normal(size=(3, 6, 8))
    offsets, rows = [1, 3, 3, 6], np.array([9, 7, 2, 0, 11, 5, 4])
    out, _ = bf16_linear.grouped(x, w, offsets, rows, 3)
    assert np.isnan(out[0]).all() and np.isnan(out[6]).all()
    assert np.allclose(out[1:3], x[[2, 0]] @ w[0].T) and np.allclose(out[3:6], x[[0, 3, 1]] @ w[2].T)


def test_experts_against_every_expert_on_every_token():
    rng = np.random.default_rng(2)
    T, H, I, E, k = 7, 8, 4, 5, 3
    q = lambda v: bf16.decode(bf16.encode(v))                                        # noqa: E731
    x, w1, w2 = q(rng.normal(size=(T, H))), q(rng.normal(size=(E, 2 * I, H))), q(rng.normal(size=(E, H, I)))
    ids = rng.integers(-1, E + 1, size=(T, k))
    ids[0] = 2
    wt = rng.normal(size=(T, k))
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                v = w1[ids[t, j]] @ x[t]
                h = q(v[:I] / (1 + np.exp(-v[:I])) * v[I:])
                want[t] += wt[t, j] * q(w2[ids[t, j]] @ h)
    assert np.allclose(bf16_linear.experts(x, ids, wt, w1, w2), want, rtol=1e-9, atol=1e-12)
    assert np.array_equal(bf16_linear.experts(x, np.full((T, k), -1), wt, w1, w2), np.zeros((T, H)))


def test_post_norm_closed_forms():
    x, r = np.array([[3.0, -4.0]]), np.array([[10.0, 20.0]])
    total, h, bound = bf16_linear.post_norm(x, r, False, 2.0 ** -60, [1.0, 2.0], np.array([[0.5]]), 2.0)
    rms = math.sqrt(12.5)
    assert np.allclose(total, [[10 + 3 / rms, 20 - 8 / rms]], rtol=1e-14) and np.all(bound < 1e-13)
    assert np.array_equal(h, total.astype(np.float32).astype(np.float64))
    assert np.array_equal(bf16_linear.post_norm(x, r, True, 1e-6)[1], [[13.0, 16.0]])
    assert bf16_linear.round_stream([1 + 2.0 ** -8], True)[0] == 1.0                  # a tie of bfloat16
