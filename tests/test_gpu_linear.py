"""GPU tier: moe_w4a4_linear against the fp64 oracle.

Tolerance: oracle.linear.sum_error (the matrix cores' sums), then half a step
of the output's type: 2^-8 (bfloat16), 2^-24 (float32) of the value."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from block_scaled_fp4_pre_amd.layer import W4A4Linear
from oracle import bf16, linear, mxfp4
from tests import fp8_mfma_model
from tests.gpu_support import dev, dev_bf16, log

pytestmark = pytest.mark.gpu

MX4, FP8 = _lib.MOE_MMA_MXF4_X_MXF4, _lib.MOE_MMA_FP8_X_MXF4
TYPES = pytest.mark.parametrize("mma", [MX4, FP8], ids=["mxf4xmxf4", "fp8xfp4"])


def tokens(T, K, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, K)) * np.exp(0.5 * rng.normal(size=K)) * np.exp(0.3 * rng.normal(size=(T, 1)))
    return bf16.encode(x.astype(np.float32).astype(np.float64))


def weights(N, K, seed):
    return mxfp4.quantize_packed((0.02 * np.random.default_rng(seed).normal(size=(N, K))).astype(np.float32))


def make_linear(K, N, max_tokens, mma, wc, ws):
    lin = W4A4Linear(K, N, max_tokens, mma_type=mma)
    lin.prepared.fill_(0xA5)                      # the padding is the library's to write
    lin.workspace.fill_(0xA5)
    lin.load_canonical(dev(wc), dev(ws))
    return lin


def reference(x, wc, ws, mma, addend=None):
    c, s = linear.quantize_tokens(bf16.decode(x), mma == FP8)
    return (c, s) + linear.linear(c, s, wc, ws, mma == FP8, addend)


def close(got, ref, mag, K, mma, f32=False):
    err = np.abs(got - ref)
    tol = linear.sum_error(mag, K, mma == FP8)
    tol = tol + (np.abs(ref) + tol) * (2.0 ** -24 if f32 else 2.0 ** -8)
    assert np.all(np.isfinite(got))
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:4])


def run(lin, x, T, N, dtype=torch.bfloat16, addend=None, quantized=None):
    """The call on rows [0, T) of a larger buffer whose other rows must stay."""
    buf = torch.full((T + 2, N), 77.0, dtype=dtype, device="cuda")
    if quantized is None:
        lin.forward(dev_bf16(x), out=buf[:T], addend=addend)
    else:
        lin.forward_quantized(*(dev(q) for q in quantized), out=buf[:T], addend=addend)
    torch.cuda.synchronize()
    assert torch.all(buf[T:] == 77.0)
    return buf[:T]


SIZES = [(1, 32, 1), (1, 64, 16), (1, 4096, 4096), (2, 96, 17), (3, 128, 64), (8, 160, 100), (15, 2048, 65), (16, 2080, 256),
         (17, 1056, 257), (31, 4096, 130), (32, 512, 1111), (33, 8192, 48), (48, 96, 2048), (63, 1024, 63),
         (64, 4096, 512), (65, 256, 300), (100, 3200, 1023), (128, 128, 128), (130, 416, 515), (255, 2048, 255),
         (256, 1024, 1024), (257, 32, 4096), (300, 1056, 1111), (513, 640, 260), (1030, 4096, 520)]


@TYPES
@pytest.mark.parametrize("T,K,N", SIZES)
def test_sizes(T, K, N, mma):
    log(f"[test] linear T {T} K {K} N {N} mma {mma}")
    x, (wc, ws) = tokens(T, K, T + K), weights(N, K, N)
    lin = make_linear(K, N, T, mma, wc, ws)
    c, s, ref, mag = reference(x, wc, ws, mma)
    got = run(lin, x, T, N)
    close(got.double().cpu().numpy(), ref, mag, K, mma)
    again = run(lin, x, T, N, quantized=(c, s))
    assert torch.equal(got, again)                # from tokens quantized before: the same bits
    f32 = run(lin, x, T, N, dtype=torch.float32)
    close(f32.double().cpu().numpy(), ref, mag, K, mma, f32=True)
    assert torch.equal(f32.to(torch.bfloat16), got)


@TYPES
@pytest.mark.parametrize("T,K,N", [(1, 512, 100), (16, 2048, 512), (40, 96, 77), (300, 1056, 260), (600, 512, 1024)])
def test_addend_apart_and_in_place(T, K, N, mma):
    log(f"[test] linear addend T {T} K {K} N {N} mma {mma}")
    x, (wc, ws) = tokens(T, K, 5), weights(N, K, 6)
    add = tokens(T, N, 7)
    lin = make_linear(K, N, T + 9, mma, wc, ws)   # a workspace for more tokens than the call's
    _, _, ref, mag = reference(x, wc, ws, mma, bf16.decode(add))
    got = run(lin, x, T, N, addend=dev_bf16(add))
    close(got.double().cpu().numpy(), ref, mag + np.abs(bf16.decode(add)), K, mma)
    out = dev_bf16(add)
    lin.forward(dev_bf16(x), out=out, addend=out)
    torch.cuda.synchronize()
    assert torch.equal(out, got)
    f32 = run(lin, x, T, N, dtype=torch.float32, addend=dev_bf16(add))
    assert torch.equal(f32.to(torch.bfloat16), got)


@TYPES
def test_scales_at_their_ends(mma):
    """Tokens of zeros, subnormals, and rows 2^+-60 apart; weights with scale
    bytes 0 and near the largest: exact powers of two throughout."""
    log(f"[test] linear extreme scales mma {mma}")
    T, K, N = 20, 256, 48
    x = tokens(T, K, 8)
    v = bf16.decode(x)
    v[0] = 0
    v[1] *= 2.0 ** 60
    v[2] *= 2.0 ** -60
    v[3, 32:] = 0
    v[4, :32] = 0
    v[5] = 2.0 ** -130
    x = bf16.encode(v)
    wc, ws = weights(N, K, 9)
    ws[0], wc[0] = 0, 0                           # a row of zeros as the quantizer writes it
    ws[1] = 127 + 40
    ws[2] = 127 - 60
    lin = make_linear(K, N, T, mma, wc, ws)
    _, _, ref, mag = reference(x, wc, ws, mma)
    got = run(lin, x, T, N, dtype=torch.float32).double().cpu().numpy()
    tol = linear.sum_error(mag, K, mma == FP8)
    assert np.all(np.abs(got - ref) <= tol + (np.abs(ref) + tol) * 2.0 ** -24 + 2.0 ** -149)
    assert np.all(got[0] == 0) and np.all(got[:, 0] == 0)


@TYPES
def test_one_set_of_weights_at_several_capacities(mma):
    log(f"[test] linear with_capacity mma {mma}")
    K, N = 1024, 640
    wc, ws = weights(N, K, 10)
    base = W4A4Linear(K, N, 1, mma_type=MX4)
    w = mxfp4.dequantize(wc, ws).astype(np.float32)
    base.load_fp32(w)                             # on the format's grid: quantizes to the same values
    x = tokens(200, K, 11)
    big = base.with_capacity(200, mma_type=mma)
    small = base.with_capacity(7, mma_type=mma)
    _, _, ref, mag = reference(x, wc, ws, mma)
    a = run(big, x, 200, N).double().cpu().numpy()
    close(a, ref, mag, K, mma)
    b = run(small, x[:7], 7, N).double().cpu().numpy()
    close(b, ref[:7], mag[:7], K, mma)
    with pytest.raises(_lib.MoeError) as ei:
        small.forward(dev_bf16(x[:8]))
    assert ei.value.status == _lib.MOE_ECAPACITY
    assert small.forward(torch.empty((0, K), dtype=torch.bfloat16, device="cuda")).shape == (0, N)


@TYPES
def test_repeats_give_the_same_bits(mma):
    log(f"[test] linear determinism mma {mma}")
    for T, K, N in ((1, 4096, 4096), (16, 4096, 1024), (64, 8192, 512), (777, 1024, 1536)):
        x, (wc, ws) = tokens(T, K, 12), weights(N, K, 13)
        lin = make_linear(K, N, T, mma, wc, ws)
        first = lin.forward(dev_bf16(x))
        for _ in range(5):
            assert torch.equal(lin.forward(dev_bf16(x)), first)


# what launch_ops.h's linear_plan sends to each tile kernel, ragged on every side
TILED = [(500, 288, 3001, "64 tokens"), (257, 32, 4096, "64 tokens"), (70, 1056, 10000, "64 tokens"),
         (1100, 160, 2050, "128 tokens"), (70, 416, 20001, "128 tokens"), (2000, 640, 2048, "128 tokens"),
         (4100, 96, 4097, "256 rows"), (16000, 416, 1030, "256 rows"), (300, 288, 50000, "256 rows")]


@TYPES
@pytest.mark.parametrize("T,K,N,plan", TILED, ids=lambda v: str(v))
def test_tile_kernels(T, K, N, plan, mma):
    t64, t128, n128, n256 = -(-T // 64), -(-T // 128), -(-N // 128), -(-N // 256)
    assert plan == ("64 tokens" if 128 < t64 * n128 <= 256 else "256 rows" if t128 * n256 >= 512 else "128 tokens")
    log(f"[test] linear T {T} K {K} N {N} mma {mma}: {plan}")
    x, (wc, ws), add = tokens(T, K, 20), weights(N, K, 21), tokens(T, N, 22)
    lin = make_linear(K, N, T, mma, wc, ws)
    c, s, ref, mag = reference(x, wc, ws, mma)
    got = run(lin, x, T, N)
    close(got.double().cpu().numpy(), ref, mag, K, mma)
    assert torch.equal(run(lin, x, T, N, quantized=(c, s)), got)
    f32 = run(lin, x, T, N, dtype=torch.float32)
    close(f32.double().cpu().numpy(), ref, mag, K, mma, f32=True)
    a = bf16.decode(add)
    plus = run(lin, x, T, N, addend=dev_bf16(add))
    close(plus.double().cpu().numpy(), ref + a, mag + np.abs(a), K, mma)
    plus32 = run(lin, x, T, N, dtype=torch.float32, addend=dev_bf16(add))
    assert torch.equal(plus32.to(torch.bfloat16), plus)
    again = run(lin, x, T, N)
    assert torch.equal(again, got)


@TYPES
@pytest.mark.parametrize("T,K,N", [(4, 8192, 100), (16, 8192, 64), (16, 8160, 33), (3, 8224, 70), (16, 16384, 48),
                                   (2, 65536, 33), (40, 65536, 20)])
def test_long_rows(T, K, N, mma):
    """Up to and past what the decode kernel holds in LDS (64 K steps), and the longest K."""
    log(f"[test] linear T {T} K {K} N {N} mma {mma}")
    x, (wc, ws) = tokens(T, K, 23), weights(N, K, 24)
    lin = make_linear(K, N, T, mma, wc, ws)
    c, s, ref, mag = reference(x, wc, ws, mma)
    got = run(lin, x, T, N)
    close(got.double().cpu().numpy(), ref, mag, K, mma)
    assert torch.equal(run(lin, x, T, N, quantized=(c, s)), got)


@TYPES
@pytest.mark.parametrize("T", [5, 70, 1100])
def test_a_token_that_is_not_finite_leaves_the_others_alone(T, mma):
    log(f"[test] linear with non-finite tokens T {T} mma {mma}")
    K, N = 256, 2050
    x, (wc, ws) = tokens(T, K, 25), weights(N, K, 26)
    lin = make_linear(K, N, T, mma, wc, ws)
    clean = run(lin, x, T, N)
    bad = x.copy()
    bad[1, 7], bad[3, 200] = 0x7FC0, 0x7F80
    got = run(lin, bad, T, N)
    keep = [t for t in range(T) if t not in (1, 3)]
    assert torch.equal(got[keep], clean[keep])


def test_offsets_past_32_bits():
    """Tokens of more than 2^32 bytes, and weights of more than 2^32 bytes of
    codes: the last tokens and rows against the oracle."""
    log("[test] linear with offsets past 32 bits")
    T, K, N = 600_001, 4096, 24
    wc, ws = weights(N, K, 27)
    lin = make_linear(K, N, T, FP8, wc, ws)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    tail = tokens(70, K, 28)
    x[-70:] = dev_bf16(tail)
    out = lin.forward(x)
    _, _, ref, mag = reference(tail, wc, ws, FP8)
    close(out[-70:].double().cpu().numpy(), ref, mag, K, FP8)
    assert torch.count_nonzero(out[:-70]).item() == 0
    del x, out, lin
    K, N = 16384, 600_003
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // 32), 120, dtype=torch.uint8, device="cuda")
    wc, ws = weights(40, K, 29)
    codes[-40:], scales[-40:] = dev(wc), dev(ws)
    lin = W4A4Linear(K, N, 20, mma_type=MX4)
    lin.load_canonical(codes, scales)
    for T in (2, 20):
        x = tokens(T, K, 30)
        out = lin.forward(dev_bf16(x))
        _, _, ref, mag = reference(x, wc, ws, MX4)
        close(out[:, -40:].double().cpu().numpy(), ref, mag, K, MX4)
        assert torch.count_nonzero(out[:, :-40]).item() == 0


@TYPES
def test_first_call_of_a_kernel_inside_a_capture(mma):
    """A call whose launch limits were not raised before is captured, replayed
    and equals the eager call."""
    log(f"[test] linear captured first, mma {mma}")
    K, N = 8192, 128
    wc, ws = weights(N, K, 31)
    lin = make_linear(K, N, 16, mma, wc, ws)
    x = dev_bf16(tokens(16, K, 32))
    out = torch.zeros((16, N), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.forward(x, out=out)
    for seed in (33, 34, 35):
        x.copy_(dev_bf16(tokens(16, K, seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, lin.forward(x))


@TYPES
@pytest.mark.parametrize("T", [3, 40, 1100])
def test_subnormal_outputs(T, mma):
    """Sums below 2^-126: the bfloat16 result is on its subnormal grid (2^-133 apart)."""
    log(f"[test] linear subnormal outputs T {T} mma {mma}")
    K, N = 64, 2050
    v = bf16.decode(tokens(T, K, 36)) * 2.0 ** -60
    x = bf16.encode(v)
    wc, ws = weights(N, K, 37)
    ws = (ws.astype(np.int32) - 63).astype(np.uint8)
    lin = make_linear(K, N, T, mma, wc, ws)
    _, _, ref, mag = reference(x, wc, ws, mma)
    assert np.mean(np.abs(ref) < 2.0 ** -126) > 0.4                   # (of the case: enough of them are subnormal)
    got = run(lin, x, T, N).double().cpu().numpy()
    tol = linear.sum_error(mag, K, mma == FP8) + 2.0 ** -149          # fp32 sums may be subnormal too
    assert np.all(np.abs(got - ref) <= tol + np.maximum(np.abs(ref) * 2.0 ** -8, 2.0 ** -134) * (1 + 2.0 ** -8))
    assert np.count_nonzero(got) > got.size / 2


@TYPES
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,N0", [(5, 264), (90, 264), (1100, 1000), (2100, 1096), (8192, 2032)])
def test_rows_of_any_length(T, N0, dtype, mma):
    """Rows at every remainder of eight values, through each kernel, with an
    addend: the columns' bits are those of rows that are aligned, and the rows'
    own last values are the last ones written."""
    log(f"[test] linear rows T {T} N {N0} {dtype} mma {mma}")
    K = 96
    x, (wc, ws), add = tokens(T, K, 31), weights(N0 + 8, K, 32), tokens(T, N0 + 8, 33)
    lin = make_linear(K, N0 + 8, T, mma, wc, ws)
    _, _, ref, mag = reference(x, wc, ws, mma, bf16.decode(add))
    whole = run(lin, x, T, N0 + 8, dtype=dtype, addend=dev_bf16(add)).clone()
    close(whole.double().cpu().numpy(), ref, mag + np.abs(bf16.decode(add)), K, mma, f32=dtype == torch.float32)
    for N in range(N0 + 1, N0 + 8):
        lin = make_linear(K, N, T, mma, np.ascontiguousarray(wc[:N]), np.ascontiguousarray(ws[:N]))
        got = run(lin, x, T, N, dtype=dtype, addend=dev_bf16(np.ascontiguousarray(add[:, :N])))
        assert torch.equal(got, whole[:, :N]), N


# on either side of what launch_ops.h's linear_plan sends to the decode kernel
FEW = [(1, 8192, 100), (1, 8160, 33), (1, 4128, 4096), (1, 4128, 4097), (1, 8224, 64), (2, 4128, 64), (1, 4096, 8200),
       (8, 4096, 5000), (9, 4096, 4100), (16, 2048, 4100), (16, 4096, 4096), (16, 4064, 4112), (16, 2080, 16)]


@TYPES
@pytest.mark.parametrize("T,K,N", FEW)
def test_few_tokens(T, K, N, mma):
    log(f"[test] linear few T {T} K {K} N {N} mma {mma}")
    x, (wc, ws), add = tokens(T, K, 41), weights(N, K, 42), tokens(T, N, 43)
    lin = make_linear(K, N, T, mma, wc, ws)
    c, s, ref, mag = reference(x, wc, ws, mma)
    got = run(lin, x, T, N)
    close(got.double().cpu().numpy(), ref, mag, K, mma)
    assert torch.equal(run(lin, x, T, N, quantized=(c, s)), got)
    a = bf16.decode(add)
    plus = run(lin, x, T, N, dtype=torch.float32, addend=dev_bf16(add))
    close(plus.double().cpu().numpy(), ref + a, mag + np.abs(a), K, mma, f32=True)


# one size for each kernel that needs more LDS than a launch has by default
CAPTURED_FIRST = [(1, 8192, 100, "decode"), (500, 288, 3001, "64 tokens"), (2000, 640, 2048, "128 tokens"),
                  (4100, 96, 4097, "256 rows")]
FRESH_PROCESS = """
import sys, torch
sys.path.insert(0, {root!r})
from tests.test_gpu_linear import CAPTURED_FIRST, FP8, MX4, dev_bf16, make_linear, tokens, weights
for mma in (MX4, FP8):
    for T, K, N, plan in CAPTURED_FIRST:
        lin = make_linear(K, N, T, mma, *weights(N, K, 51))
        xs = [dev_bf16(tokens(T, K, s)) for s in (52, 53)]
        x, out = xs[0].clone(), torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lin.forward(x, out=out)              # the process's first call of this kernel
        for i in (1, 0, 1):
            x.copy_(xs[i])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, lin.forward(xs[i])), (mma, plan)
        assert torch.count_nonzero(out).item() > T * N // 2
        print("captured first:", mma, plan, flush=True)
"""


def test_every_kernels_first_call_inside_a_capture():
    """In a process of its own, where no launch limit was raised before."""
    log("[test] linear kernels captured first, in a fresh process")
    for T, K, N, plan in CAPTURED_FIRST:         # launch_ops.h's linear_plan
        steps, t64, t128, n128, n256 = -(-K // 128), -(-T // 64), -(-T // 128), -(-N // 128), -(-N // 256)
        if plan == "decode":                     # more than 64 KiB of operands and sums in LDS
            assert 32 < steps <= 64 and T == 1 and N <= 256 * 16 and steps * (1024 + 64) + 16384 > 65536
        else:
            assert T > 16 and t64 * n128 > 128
            assert plan == ("64 tokens" if t64 * n128 <= 256 else "256 rows" if t128 * n256 >= 512 else "128 tokens")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-u", "-c", FRESH_PROCESS.format(root=root)], cwd=root, capture_output=True,
                       text=True, timeout=110)
    print(r.stdout)
    assert r.returncode == 0 and r.stdout.count("captured first:") == 2 * len(CAPTURED_FIRST), r.stdout + r.stderr


@pytest.mark.parametrize("T,K,N", [(3, 128, 100), (16, 1024, 40), (40, 256, 70), (64, 1024, 33), (500, 256, 3001), (1100, 128, 2050),
                                   (4100, 128, 4097)])
def test_e4m3_sums_against_the_matrix_cores_model(T, K, N):
    """float32 outputs of E4M3 tokens against tests/fp8_mfma_model.py: which bits
    a matrix instruction drops is known, so what is left is the bound of its
    block alignment and a half step (2^-24) of every partial sum."""
    log(f"[test] linear T {T} K {K} N {N} E4M3 against the model")
    x, (wc, ws) = tokens(T, K, 54), weights(N, K, 55)
    lin = make_linear(K, N, T, FP8, wc, ws)
    got = run(lin, x, T, N, dtype=torch.float32).double().cpu().numpy()
    rows = np.unique(np.r_[0:min(T, 20), T - min(T, 20):T])
    c, s = linear.quantize_tokens(bf16.decode(x[rows]), True)
    w = mxfp4.unpack(wc)
    ref = np.zeros((len(rows), N))
    mag, tol = np.zeros_like(ref), np.zeros_like(ref)
    for k in range(K // 128):                    # each step's sum by itself, exact before its one rounding
        step, bound = fp8_mfma_model.gemm(c[:, 128 * k:128 * k + 128], s[:, 4 * k:4 * k + 4], w[:, 128 * k:128 * k + 128],
                                          ws[:, 4 * k:4 * k + 4], with_bound=True)
        ref += step
        mag += np.abs(step)
        # the model's bound for a step whose scales differ, and the step's own rounding
        tol += bound + np.abs(step) * 2.0 ** -24
    # alignment with the running sum (the model's 2^-22) and the rounding into it, and the
    # up to eight partial sums of the kernels that split K: none is above mag
    tol += ((K // 128 - 1) * (2.0 ** -22 + 2.0 ** -24) + 8 * 2.0 ** -24) * mag + 2.0 ** -149
    err = np.abs(got[rows] - ref)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:4])
