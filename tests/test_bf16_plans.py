"""CPU tier: the sizes of tests/bf16_plans.py reach every kernel of the bfloat16 linears, and
their whole operands show a sum that is not the product's."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests.bf16_plans import CASES, IDS, PLANS, largest, offsets, whole
from tests.test_abi_ops_cpu import CSRC, HERE, ROOT

ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path_factory.mktemp("plan") / "bf16_plan_check"
    cmd = [gxx, "-std=c++17", "-O2", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"), "-I",
           os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(HERE, "bf16_plan_check.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ)
    env.pop("LD_PRELOAD", None)

    def ask(text):
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, env=env, timeout=120)
        assert r.returncode == 0, r.stderr
        return r.stdout.split("\n")[:-1]
    return ask


def test_every_size_takes_the_kernel_of_its_row(rule):
    got = rule("".join(f"{T} {N} {K} {groups} {int(gated)}\n" for _, gated, groups, T, K, N in CASES))
    assert [(PLANS[int(p)], *c[1:]) for p, c in zip(got, CASES)] == CASES


def test_every_kernel_that_the_rule_reaches_has_a_size(rule):
    reached = {tuple(map(int, line.split())) for line in rule("sweep\n")}
    assert reached == {(PLANS.index(plan), int(gated), int(groups > 0)) for plan, gated, groups, *_ in CASES}
    header = open(os.path.join(CSRC, "launch_bf16.h")).read()
    names = header[header.index("enum Bf16Plan {"):]
    assert names[:names.index("}")].count("k") == len(PLANS)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_whole_operands_show_a_wrong_sum(case):
    """On some of the rows and columns: without the last 8 values of K, without its last step,
    with two pieces changed over, and in sums of 12 bits fewer, nearly every output is another
    number (with operands of -1, 0 and 1, 8 products now and then add up to 0)."""
    _, _, _, T, K, N = case
    rng = np.random.default_rng([T, K, N])
    for most, share in ((largest(K), 0.97), (1, 0.6)):
        assert K * most * most <= 2 ** 24
        x, w = whole(rng, (min(T, 64), K), most), whole(rng, (min(N, 64), K), most)
        v, last = x @ w.T, (K - 1) // 64 * 64
        moved = w.copy()
        moved[:, :8], moved[:, 8:16] = w[:, 8:16], w[:, :8]
        for wrong in (x[:, :-8] @ w[:, :-8].T, x[:, :last] @ w[:, :last].T, x @ moved.T):
            assert (wrong != v).mean() > share
        if most > 1:
            assert (v % 256 != 0).mean() > share


def test_groups_are_uneven():
    for _, _, groups, T, _, _ in CASES:
        if groups:
            sizes = np.diff(offsets(T, groups))
            assert sizes.sum() == T and sizes.min() == 0 and 2 * sizes.max() >= T - groups
