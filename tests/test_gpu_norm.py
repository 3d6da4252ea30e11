"""GPU tier: moe_w4a4_add_rmsnorm against the fp64 oracle, for every launch
shape of the kernel, residual type and activation format.

Tolerances: the device sums and multiplies in fp64 in another order than the
oracle, at most C + 8 roundings of 2^-53 relative, so y lies between the
roundings (to float32, then bfloat16) of n * (1 - d) and n * (1 + d) with d =
(C + 8) * 2^-53 -- the same bfloat16 but next to a border.  The residual sum is
one exact rounding, and codes and scales are those the oracle's quantizer makes
of the device's y, byte for byte."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from oracle import bf16, mxfp4, mxfp8, norm, nvfp4
from tests.gpu_support import dev, dev_bf16, host_bits, log

pytestmark = pytest.mark.gpu

EPS = 1e-6
MX4, FP8, NV4 = _lib.MOE_MMA_MXF4_X_MXF4, _lib.MOE_MMA_FP8_X_MXF4, _lib.MOE_MMA_NVF4_X_NVF4


def make(rows, cols, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=cols)) * scale
    return bf16.encode(x.astype(np.float32).astype(np.float64))


def check(x, r, res, weight, w_bf16, mma, want_y=True, g=2.0 ** -9, inplace=False, eps=EPS):
    """x bf16 bits; r fp64 values or None; res 'bf16' | 'f32' | None; mma None: no codes."""
    rows, cols = x.shape
    xd = dev_bf16(x)
    wd = dev_bf16(bf16.encode(weight)) if w_bf16 else dev(weight.astype(np.float32))
    wv = bf16.decode(bf16.encode(weight)) if w_bf16 else weight.astype(np.float32).astype(np.float64)
    rd = ro = None
    h = bf16.decode(x)
    if res is not None:
        rd = dev_bf16(bf16.encode(r)) if res == "bf16" else dev(r.astype(np.float32))
        rv = bf16.decode(bf16.encode(r)) if res == "bf16" else r.astype(np.float32).astype(np.float64)
        ro = rd if inplace else torch.full_like(rd, float("nan"))
        h = norm.residual_sum(h, rv, res == "bf16")
    y = (xd if inplace else torch.full_like(xd, float("nan"))) if want_y else None
    codes = scales = None
    if mma is not None:
        codes = torch.full((rows + 1, cols if mma == FP8 else cols // 2), 0xA5, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows + 1, cols // (16 if mma == NV4 else 32)), 0xA5, dtype=torch.uint8, device="cuda")
    _lib.moe_w4a4_add_rmsnorm(xd, rd, wd, eps, residual_out=ro, y=y, codes=None if codes is None else codes[:rows],
                              scales=None if scales is None else scales[:rows], mma_type=mma or 0, tensor_scale=g)
    torch.cuda.synchronize()
    if res == "bf16":
        assert np.array_equal(host_bits(ro), bf16.encode(h))
    elif res == "f32":
        assert np.array_equal(ro.cpu().numpy().astype(np.float64), h)
    n, d = norm.rmsnorm(h, wv, eps), (cols + 8) * 2.0 ** -53
    lo, hi = norm.round_y(n * (1 - d)), norm.round_y(n * (1 + d))
    if want_y:
        got = host_bits(y)
        assert np.all((got == lo) | (got == hi)), int(np.sum((got != lo) & (got != hi)))
    else:
        assert np.array_equal(lo, hi)                      # no value next to a border in this case
        got = lo
    if mma is not None:
        assert torch.all(codes[rows] == 0xA5) and torch.all(scales[rows] == 0xA5)     # rows behind the last
        v = bf16.decode(got)
        c, s = (nvfp4.quantize_packed(v, g) if mma == NV4 else (mxfp8 if mma == FP8 else mxfp4).quantize_packed(v))
        assert np.array_equal(codes[:rows].cpu().numpy(), c) and np.array_equal(scales[:rows].cpu().numpy(), s)


# every launch shape's smallest and largest width, and a ragged one inside
@pytest.mark.parametrize("cols", [32, 96, 512, 544, 1024, 1056, 2048, 2080, 4096, 4128, 7200, 8192, 8224, 16384, 16416,
                                  32768, 32800, 65536])
@pytest.mark.parametrize("mma", [MX4, FP8, NV4], ids=["mxfp4", "mxfp8", "nvfp4"])
def test_every_width_and_format(cols, mma):
    log(f"[test] norm cols {cols} format {mma}")
    rng = np.random.default_rng(cols)
    rows = 1 if cols > 16384 else 5
    check(make(rows, cols, 1), 3 * rng.normal(size=(rows, cols)), "bf16", 1 + 0.1 * rng.normal(size=cols), False, mma)


@pytest.mark.parametrize("res", [None, "bf16", "f32"])
@pytest.mark.parametrize("w_bf16", [False, True])
@pytest.mark.parametrize("cols", [256, 4096])
def test_residual_and_weight_types(res, w_bf16, cols):
    log(f"[test] norm residual {res}, bf16 weight {w_bf16}, cols {cols}")
    rng = np.random.default_rng(7)
    r = 3 * rng.normal(size=(9, cols))
    w = 1 + 0.1 * rng.normal(size=cols)
    check(make(9, cols, 2), r, res, w, w_bf16, FP8)
    check(make(9, cols, 3), r, res, w, w_bf16, None)                  # y alone
    check(make(9, cols, 4), r, res, w, w_bf16, MX4, want_y=False)     # codes alone


@pytest.mark.parametrize("res", [None, "bf16", "f32"])
@pytest.mark.parametrize("cols", [512, 8192])
def test_in_place(res, cols):
    log(f"[test] norm in place, residual {res}, cols {cols}")
    rng = np.random.default_rng(8)
    check(make(33, cols, 5), rng.normal(size=(33, cols)), res, 1 + 0.1 * rng.normal(size=cols), False, FP8, inplace=True)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 63, 64, 1000, 2048, 4100])
@pytest.mark.parametrize("cols", [64, 2048])
def test_row_counts(rows, cols):
    log(f"[test] norm rows {rows} cols {cols}")
    check(make(rows, cols, rows), None, None, np.ones(cols), False, FP8)


def test_extreme_values():
    """Rows of zeros, one value only, squares that pass float32's range at both
    ends, subnormals, and signed zeros."""
    log("[test] norm extreme values")
    cols = 128
    x = make(8, cols, 11)
    x[0] = 0
    x[1] = 0
    x[1, 77] = bf16.encode(np.array([1.0]))[0]
    x[2] = bf16.encode(np.full(cols, 2.0 ** 100))
    x[3] = bf16.encode(np.full(cols, 2.0 ** -100))
    x[4] = np.arange(cols)                                             # subnormals
    x[5] = 0x8000                                                      # -0
    x[6] = bf16.encode(np.ldexp(1.0, np.arange(cols) % 120 - 60))
    w = np.ones(cols)
    for mma in (MX4, FP8):
        check(x, None, None, w, False, mma)
    check(x, None, None, w, False, FP8, eps=2.0 ** -140)
    check(x, None, None, 2.0 ** np.arange(-64, 64), False, FP8)


def test_a_row_with_infinities_leaves_the_others_alone():
    log("[test] norm with a non-finite row")
    x = make(6, 256, 12)
    clean = [torch.empty((6, 256), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    codes = [torch.zeros((6, 256), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((6, 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    bad = x.copy()
    bad[2, 5], bad[2, 9] = 0x7F80, 0x7FC0
    for i, v in enumerate((x, bad)):
        _lib.moe_w4a4_add_rmsnorm(dev_bf16(v), None, torch.ones(256, device="cuda"), EPS, y=clean[i], codes=codes[i],
                                  scales=scales[i], mma_type=FP8)
    torch.cuda.synchronize()
    keep = [0, 1, 3, 4, 5]
    for a, b in (clean, codes, scales):
        assert torch.equal(a[keep], b[keep])
    assert not torch.isfinite(clean[1][2]).all()


def test_no_rows_and_equals_the_layers_own_quantizer():
    log("[test] norm: no rows; codes equal moe_w4a4_quantize of y")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    _lib.moe_w4a4_add_rmsnorm(e, None, torch.ones(64, device="cuda"), EPS, y=e)
    x = dev_bf16(make(40, 4096, 13))
    y, c, s = torch.empty_like(x), torch.empty((40, 2048), dtype=torch.uint8, device="cuda"), \
        torch.empty((40, 128), dtype=torch.uint8, device="cuda")
    _lib.moe_w4a4_add_rmsnorm(x, None, torch.ones(4096, device="cuda"), EPS, y=y, codes=c, scales=s, mma_type=MX4)
    c2, s2 = torch.empty_like(c), torch.empty_like(s)
    _lib.moe_w4a4_quantize(y, c2, s2)
    torch.cuda.synchronize()
    assert torch.equal(c, c2) and torch.equal(s, s2)


def test_offsets_past_32_bits():
    """More than 2^31 values in all: the last rows against the oracle."""
    log("[test] norm with offsets past 32 bits")
    rows, cols = 524_299, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = make(9, cols, 14)
    x[-9:] = dev_bf16(tail)
    y = torch.empty_like(x)
    codes = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device="cuda")
    _lib.moe_w4a4_add_rmsnorm(x, None, torch.ones(cols, device="cuda"), EPS, y=y, codes=codes, scales=scales, mma_type=FP8)
    torch.cuda.synchronize()
    n, d = norm.rmsnorm(bf16.decode(tail), np.ones(cols), EPS), (cols + 8) * 2.0 ** -53
    got = host_bits(y[-9:])
    assert np.all((got == norm.round_y(n * (1 - d))) | (got == norm.round_y(n * (1 + d))))
    c, s = mxfp8.quantize_packed(bf16.decode(got))
    assert np.array_equal(codes[-9:].cpu().numpy(), c) and np.array_equal(scales[-9:].cpu().numpy(), s)
    assert torch.count_nonzero(y[:-9]).item() == 0 and torch.count_nonzero(codes[:-9]).item() == 0


@pytest.mark.parametrize("cols", [512, 4096, 65536])
def test_captured_and_replayed(cols):
    log(f"[test] norm captured, cols {cols}")
    x, r = (dev_bf16(make(3, cols, s)) for s in (15, 16))
    w = torch.ones(cols, device="cuda")
    y, ro = torch.empty_like(x), torch.empty_like(r)
    c, s = torch.empty((3, cols // 2), dtype=torch.uint8, device="cuda"), \
        torch.empty((3, cols // 32), dtype=torch.uint8, device="cuda")
    call = lambda: _lib.moe_w4a4_add_rmsnorm(x, r, w, EPS, residual_out=ro, y=y, codes=c, scales=s, mma_type=MX4)  # noqa: E731
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (17, 18, 19):
        x.copy_(dev_bf16(make(3, cols, seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, ro, c, s)]
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, ro, c, s)))


def test_subnormal_sums_and_outputs():
    """bfloat16 results below 2^-126, in the residual and in y."""
    log("[test] norm subnormal results")
    rng = np.random.default_rng(20)
    x = bf16.encode(np.ldexp(rng.integers(-127, 128, size=(4, 128)).astype(np.float64), -133))
    r = np.ldexp(rng.integers(-127, 128, size=(4, 128)).astype(np.float64), -133)
    check(x, r, "bf16", np.ones(128), False, FP8)
    check(make(4, 128, 21), None, None, np.full(128, 2.0 ** -130), False, MX4)
    check(make(4, 128, 22), None, None, 2.0 ** -np.linspace(100, 148, 128).round(), False, None)


def test_more_rows_than_blocks():
    """Over 2^20 rows a workgroup takes several; the same rows give the same bits."""
    log("[test] norm with more rows than workgroups")
    rows, cols, part = (1 << 20) + 70_001, 1056, 1000
    x = dev_bf16(make(part, cols, 23)).repeat(-(-rows // part), 1)[:rows].contiguous()
    y = torch.empty_like(x)
    _lib.moe_w4a4_add_rmsnorm(x, None, torch.ones(cols, device="cuda"), EPS, y=y)
    few = torch.empty((part, cols), dtype=torch.bfloat16, device="cuda")
    _lib.moe_w4a4_add_rmsnorm(x[:part].contiguous(), None, torch.ones(cols, device="cuda"), EPS, y=few)
    torch.cuda.synchronize()
    whole = rows // part * part
    assert torch.equal(y[:whole].view(-1, part, cols).amin(0), few) and torch.equal(y[:whole].view(-1, part, cols).amax(0), few)
    assert torch.equal(y[whole:], few[:rows - whole])


# past 8192 values the row count chooses the team: both sides of the change
@pytest.mark.parametrize("rows", [256, 257, 300])
@pytest.mark.parametrize("cols,res,mma", [(8224, None, FP8), (9504, "bf16", MX4), (16384, "f32", NV4), (16352, None, None)])
def test_many_long_rows(rows, cols, res, mma):
    log(f"[test] norm long rows {rows} x {cols} residual {res} format {mma}")
    rng = np.random.default_rng(rows + cols)
    r = None if res is None else rng.normal(size=(rows, cols))
    check(make(rows, cols, cols), r, res, np.exp(0.3 * rng.normal(size=cols)), False, mma, inplace=rows == 300)


@pytest.mark.parametrize("cols", [512, 4096, 16384])
def test_y_in_the_place_of_a_bf16_residual(cols):
    log(f"[test] norm y over the residual, cols {cols}")
    x, r = dev_bf16(make(300, cols, 24)), dev_bf16(make(300, cols, 25))
    w = torch.linspace(0.5, 2.0, cols, device="cuda")
    h, y = torch.empty_like(x), torch.empty_like(x)
    _lib.moe_w4a4_add_rmsnorm(x, r, w, EPS, residual_out=h, y=y)
    h2 = torch.empty_like(x)
    _lib.moe_w4a4_add_rmsnorm(x, r, w, EPS, residual_out=h2, y=r)
    torch.cuda.synchronize()
    assert torch.equal(h2, h) and torch.equal(r, y)
