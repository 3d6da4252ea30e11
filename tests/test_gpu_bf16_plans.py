"""GPU tier: every kernel of the bfloat16 linears (tests/bf16_plans.py) on whole operands, whose
products, sums and epilogues are exact in float32 in any order: the outputs are compared
with fp64's number for number, bfloat16 ones with its rounding to nearest, ties to even.

The activations' arguments are exact there as well (operands of -1, 0 and 1, the weights'
an eighth of it), so what is left is f within 2^-20 of its value (2^-126 of a tail) and half
a step, 2^-24, each of the gate's product and the addend, then of the output's type."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from tests.bf16_plans import CASES, IDS, largest, offsets, whole
from tests.gpu_support import dev, log
from tests.test_gpu_bf16_linear import FN, SIZES

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def held(t, pad, fill=77.0):
    """t (a copy) in rows that are `pad` values wider, with two more rows behind: (all of it, the view)."""
    wide = torch.full((t.shape[0] + 2, t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    wide[:t.shape[0], :t.shape[1]] = t
    return wide, wide[:t.shape[0], :t.shape[1]]


class Product:
    """One case's call and its fp64 values."""

    def __init__(self, case, most, unit=1.0, gather=0, seed=0):
        _, self.gated, self.groups, self.T, self.K, self.N = case
        rng = np.random.default_rng([*case[2:], most, seed])
        self.rng, wide = rng, 2 * self.N if self.gated else self.N
        rows = max(1, -(-self.T // gather)) if gather else self.T
        self.x = torch.from_numpy(whole(rng, (rows, self.K), most)).cuda().to(BF)
        g = torch.Generator(device="cuda").manual_seed(seed + self.N)
        self.w = (torch.randint(-most, most + 1, (max(1, self.groups), wide, self.K), generator=g, device="cuda") * unit).to(BF)
        self.bounds = offsets(self.T, self.groups) if self.groups else np.array([0, self.T])
        self.gather = gather
        self.rows = torch.from_numpy(rng.permutation(rows * gather)[:self.T].astype(np.int32)).cuda() if gather else None

    def sums(self):
        """fp64 [T, N or 2N]."""
        x = self.x if self.rows is None else self.x[(self.rows // self.gather).long()]
        return torch.cat([x[a:b].double() @ w.double().t().contiguous()
                          for a, b, w in zip(self.bounds, self.bounds[1:], self.w)])

    def by_row(self, v):
        """[groups, n] values as [T, n]."""
        return torch.repeat_interleave(v.double(), torch.from_numpy(np.diff(self.bounds)).cuda(), 0)

    def call(self, out, **kw):
        if self.groups:
            _lib.moe_w4a4_grouped_linear_bf16(self.x, self.w, dev(self.bounds.astype(np.int32)), out, rows=self.rows,
                                              row_divisor=max(1, self.gather), gated=self.gated, **kw)
        else:
            kw = {k: v[0] if k == "bias" and v is not None else v for k, v in kw.items()}
            _lib.moe_w4a4_linear_bf16(self.x, self.w[0], out, gated=self.gated, **kw)
        torch.cuda.synchronize()

    def run(self, dtype, pad=3, **kw):
        wide, out = held(torch.zeros((self.T, self.N), dtype=dtype, device="cuda"), pad)
        self.call(out, **kw)
        assert torch.all(wide[self.T:] == 77.0) and torch.all(wide[:, self.N:] == 77.0)
        return out


def exact(got, want):
    assert torch.equal(want, want.float().double()), "the reference is not a float32: the case's operands are too large"
    bad = got != want.float().to(got.dtype)
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:4].tolist())


def sums_exact(case, gather=0):
    p = Product(case, largest(case[4]), gather=gather)
    v = p.sums()
    for dtype in (F32, BF):
        if not p.gated:
            exact(p.run(dtype), v)
            continue
        # gate * up with one of the two held at 1 by the bias: the other's sum as it is
        for half in (0, 1):
            w = p.w.clone()
            w[:, (1 - half) * p.N:(2 - half) * p.N] = 0
            bias = torch.zeros(p.w.shape[:2], device="cuda")
            bias[:, (1 - half) * p.N:(2 - half) * p.N] = 1
            p.w, kept = w, p.w
            got = p.run(dtype, bias=bias)
            p.w = kept
            exact(got, v[:, half * p.N:(half + 1) * p.N])


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_sums(case):
    log(f"[test] bf16 sums {case}")
    sums_exact(case)
    if case[2]:
        sums_exact(case, gather=3)


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_sums_of_more_sizes(T, K, N, gated):
    log(f"[test] bf16 sums T {T} K {K} N {N} gated {gated}")
    sums_exact(("", gated, 0, T, K, N))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_epilogues(case):
    """Bias, relu, gate, row scale and addend of either type, in place and apart, strided rows."""
    log(f"[test] bf16 epilogues {case}")
    p = Product(case, 1, gather=2 if case[2] else 0, seed=1)
    quarter = lambda *shape: torch.from_numpy(p.rng.integers(-64, 65, size=shape) / 4).cuda()      # noqa: E731
    v, n = p.sums(), p.N
    for fn, bias, scaled, add, dtype, in_place in (("none", F32, True, BF, BF, False), ("relu", BF, True, F32, F32, False),
                                                   ("none", BF, False, BF, BF, True), ("relu", None, True, F32, F32, True),
                                                   ("none", None, True, None, BF, False), ("relu", F32, False, BF, F32, False)):
        b = None if bias is None else quarter(*p.w.shape[:2]).to(bias)
        s = torch.from_numpy(2.0 ** p.rng.integers(-2, 3, size=p.T)).cuda().float() if scaled else None
        a = None if add is None else quarter(p.T, n).to(add)
        want = v if b is None else v + p.by_row(b)
        gate = want[:, :n] if fn == "none" else torch.clamp(want[:, :n], min=0)
        want = gate * want[:, n:] if p.gated else gate
        if s is not None:
            want = want * s.double()[:, None]
        if a is not None:
            want = want + a.double()
        kw = dict(bias=b, function=FN[fn], row_scale=s)
        if in_place:
            wide, out = held(a, 5)
            p.call(out, addend=out, **kw)
            assert torch.all(wide[p.T:] == 77.0) and torch.all(wide[:, n:] == 77.0)
        else:
            out = p.run(dtype, addend=None if a is None else held(a, 11)[1], **kw)
        exact(out, want)


FUNCTIONS = {"silu": lambda v: v * torch.sigmoid(v), "gelu": lambda v: 0.5 * v * torch.special.erfc(-v / 2 ** 0.5),
             "gelu_tanh": lambda v: v * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3))}


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_functions(case):
    log(f"[test] bf16 functions {case}")
    p = Product(case, 1, unit=0.125, seed=2)
    v, n = p.sums(), p.N
    a = torch.from_numpy(p.rng.integers(-64, 65, size=(p.T, n)) / 4).cuda().to(BF)
    up = v[:, n:] if p.gated else torch.ones((), dtype=torch.float64, device="cuda")
    for fn, function in FUNCTIONS.items():
        step = function(v[:, :n]) * up
        bound = step.abs() * (2.0 ** -20 + 2.0 ** -24) + 2.0 ** -126 * up.abs()
        for dtype, half, add in ((F32, 2.0 ** -24, None), (BF, 2.0 ** -8, a)):
            want = step if add is None else step + add.double()
            tol = bound if add is None else bound + (want.abs() + bound) * 2.0 ** -24
            tol = tol + (want.abs() + tol) * half
            err = (p.run(dtype, function=FN[fn], addend=add).double() - want).abs()
            assert bool((err <= tol).all()), (fn, float((err / tol).max()), torch.nonzero(~(err <= tol))[:4].tolist())


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_non_finite_values_stay_in_their_row_and_column(case):
    """An infinity in the first piece of K and a NaN in the last of a row that shares its tile
    (with a group, its last), and a weight row of infinities; what lies behind K in a row is not read."""
    log(f"[test] bf16 non-finite {case}")
    p = Product(case, 1, seed=3)
    want = p.sums()
    g = p.groups // 2                                        # the largest group
    rows, bad, col = slice(int(p.bounds[g]), int(p.bounds[g + 1])), int(p.bounds[g + 1]) - 1, p.N - 1
    x = torch.full((p.T, p.K + 8), float("nan"), dtype=BF, device="cuda")
    x[:, :p.K] = p.x
    p.x = x[:, :p.K]
    p.x[bad, 0], p.x[bad, p.K - 1] = float("inf"), float("nan")
    p.w[g, col] = float("inf")                               # (0 times it is a NaN)
    got = p.run(F32)
    if p.gated:
        want = want[:, :p.N] * want[:, p.N:]
    assert not torch.isfinite(got[bad]).any() and not torch.isfinite(got[rows, col]).any()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[bad] = keep[rows, col] = False
    exact(got[keep], want[keep])
