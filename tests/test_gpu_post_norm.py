"""GPU tier: moe_w4a4_post_norm against the fp64 oracle, for every launch shape, type, gate
and activation format, and a block that ends with it.

Tolerances: h is the rounding of a value within oracle.bf16_linear.post_norm's bound of the
oracle's, so it lies between the roundings of that value less and plus the bound.  y
follows from the device's h as moe_w4a4_add_rmsnorm's does (tests/test_gpu_norm.py), and
codes and scales are those the oracle's quantizer makes of the device's y, byte for byte."""
import numpy as np
import pytest
import torch

import synth
from block_scaled_fp4_pre_amd import _lib
from block_scaled_fp4_pre_amd.layer import Bf16Experts, Bf16Linear, Bf16MLP
from oracle import bf16, bf16_linear, mxfp4, mxfp8, norm, nvfp4
from tests.gpu_support import dev, dev_bf16, host_bits, layer_for, log

pytestmark = pytest.mark.gpu

EPS = 1e-6
MX4, FP8, NV4 = _lib.MOE_MMA_MXF4_X_MXF4, _lib.MOE_MMA_FP8_X_MXF4, _lib.MOE_MMA_NVF4_X_NVF4
BF = torch.bfloat16


def typed(v, f32):
    """(device tensor, fp64 values) of v in float32 or bfloat16."""
    v = np.asarray(v, np.float32)
    if f32:
        return dev(v), v.astype(np.float64)
    bits = bf16.encode(v.astype(np.float64))
    return dev_bf16(bits), bf16.decode(bits)


def check(rows, cols, seed=0, res_f32=False, w_f32=True, post=True, gate=None, gate_f32=True, scale=0.7, want_next=True,
          want_y=True, mma=None, inplace=False, x=None, r=None):
    rng = np.random.default_rng([rows, cols, seed])
    xd, xv = typed(rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=cols)) if x is None else x, False)
    rd, rv = typed(3 * rng.normal(size=(rows, cols)) if r is None else r, res_f32)
    pd = pv = gd = gv = nd = nv = None
    if post:
        pd, pv = typed(1 + 0.1 * rng.normal(size=cols), w_f32)
    if want_next:
        nd, nv = typed(1 + 0.1 * rng.normal(size=cols), w_f32)
    if gate is not None:
        gd, gv = typed(rng.random({"channel": cols, "row": (rows, 1), "full": (rows, cols)}[gate]), gate_f32)
    ro = rd if inplace else torch.full_like(rd, float("nan"))
    y = None if not (want_next and want_y) else xd if inplace else torch.full_like(xd, float("nan"))
    codes = scales = None
    g = 2.0 ** -9
    if mma is not None:
        codes = torch.full((rows + 1, cols if mma == FP8 else cols // 2), 0xA5, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows + 1, cols // (16 if mma == NV4 else 32)), 0xA5, dtype=torch.uint8, device="cuda")
    _lib.moe_w4a4_post_norm(xd, rd, ro, EPS, post_weight=pd, gate=gd, scale=scale, next_weight=nd, y=y,
                            codes=None if codes is None else codes[:rows], scales=None if scales is None else scales[:rows],
                            mma_type=mma or 0, tensor_scale=g)
    torch.cuda.synchronize()
    total, _, bound = bf16_linear.post_norm(xv, rv, not res_f32, EPS, pv, gv, scale)
    h = ro.double().cpu().numpy() if res_f32 else bf16.decode(host_bits(ro))
    lo, hi = (bf16_linear.round_stream(total + s * bound, not res_f32) for s in (-1, 1))
    # (where the step cancels the stream, more than one float32 lies between the two: the bound
    # goes by the step, a float32's distance by what is left of the sum)
    assert np.all((lo <= h) & (h <= hi)), int(np.sum((h < lo) | (h > hi)))
    if not want_next:
        return
    n, d = norm.rmsnorm(h, nv, EPS), (cols + 8) * 2.0 ** -53
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
@pytest.mark.parametrize("res_f32", [False, True], ids=["bf16", "f32"])
def test_every_width(cols, res_f32):
    log(f"[test] post_norm cols {cols} residual f32 {res_f32}")
    rows = 1 if cols > 16384 else 5
    for i, mma in enumerate((MX4, FP8, NV4, None)):
        check(rows, cols, i, res_f32, mma=mma, gate=("channel", "row", "full", None)[i])


@pytest.mark.parametrize("gate", [None, "channel", "row", "full"])
@pytest.mark.parametrize("gate_f32", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("cols", [256, 4096])
def test_gates_and_types(gate, gate_f32, post, cols):
    log(f"[test] post_norm gate {gate} f32 {gate_f32} post {post} cols {cols}")
    for res_f32 in (False, True):
        check(9, cols, 1, res_f32, w_f32=gate_f32, post=post, gate=gate, gate_f32=gate_f32, mma=FP8)
        check(9, cols, 2, res_f32, w_f32=not gate_f32, post=post, gate=gate, gate_f32=gate_f32, scale=-1.5)
        check(9, cols, 3, res_f32, post=post, gate=gate, gate_f32=gate_f32, want_next=False)       # h alone
        check(9, cols, 4, res_f32, post=post, gate=gate, gate_f32=gate_f32, want_y=False, mma=MX4)  # codes alone


@pytest.mark.parametrize("res_f32", [False, True])
@pytest.mark.parametrize("cols", [512, 8192, 16384])
def test_in_place(res_f32, cols):
    log(f"[test] post_norm in place, cols {cols}")
    check(33, cols, 5, res_f32, gate="channel", mma=FP8, inplace=True)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 63, 64, 300, 1000, 2048, 4100])
@pytest.mark.parametrize("cols", [64, 2048])
def test_row_counts(rows, cols):
    log(f"[test] post_norm rows {rows} cols {cols}")
    check(rows, cols, gate="row", mma=FP8)


def test_y_in_the_place_of_the_residual_and_h_in_the_place_of_x():
    log("[test] post_norm other places")
    rng = np.random.default_rng(1)
    x, r, w = (dev_bf16(bf16.encode(rng.normal(size=s).astype(np.float32).astype(np.float64))) for s in ((40, 4096), (40, 4096), 4096))
    h, y = torch.empty_like(x), torch.empty_like(x)
    _lib.moe_w4a4_post_norm(x, r, h, EPS, post_weight=w, next_weight=w, y=y)
    x2, r2 = x.clone(), r.clone()
    _lib.moe_w4a4_post_norm(x2, r2, x2, EPS, post_weight=w, next_weight=w, y=r2)
    torch.cuda.synchronize()
    assert torch.equal(x2, h) and torch.equal(r2, y)


def test_extreme_values():
    """Rows of zeros, squares past float32's range at both ends, a step that cancels the
    stream; a row with a NaN leaves the others alone."""
    log("[test] post_norm extreme values")
    cols = 128
    rng = np.random.default_rng(2)
    x, r = rng.normal(size=(6, cols)), rng.normal(size=(6, cols))
    x[0] = 0
    x[1] = r[1] = 0
    x[2], x[3] = 2.0 ** 100, 2.0 ** -100
    r[4] = 2.0 ** -120
    x[5] = np.float32(bf16.decode(bf16.encode(x[5].astype(np.float32).astype(np.float64))))
    r[5] = -x[5]
    check(6, cols, 0, x=x, r=r, mma=FP8)
    check(6, cols, 1, x=x, r=r, post=False, scale=1.0, gate=None, want_next=False)
    xd, rd, w = typed(x, False)[0], typed(r, True)[0], torch.ones(cols, device="cuda")
    outs = []
    for bad in (False, True):
        xi, h, y = xd.clone(), torch.empty_like(rd), torch.empty_like(xd)
        if bad:
            xi[3, 17] = float("nan")
        _lib.moe_w4a4_post_norm(xi, rd, h, EPS, post_weight=w, next_weight=w, y=y)
        outs.append((h, y))
    torch.cuda.synchronize()
    keep = [0, 1, 2, 4, 5]
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(*outs))
    assert not torch.isfinite(outs[1][0][3]).any()


def test_captured_and_on_another_stream():
    log("[test] post_norm in a graph and on another stream")
    g = torch.Generator(device="cuda").manual_seed(0)
    x, r = (torch.randn((50, 2048), generator=g, device="cuda").to(BF) for _ in range(2))
    w = torch.ones(2048, device="cuda")

    def call(a, b, h, y, stream=None):
        _lib.moe_w4a4_post_norm(a, b, h, EPS, post_weight=w, scale=0.5, next_weight=w, y=y, stream=stream)

    want = [torch.empty_like(x) for _ in range(2)]
    call(x, r, *want)
    side, got = torch.cuda.Stream(), [torch.empty_like(x) for _ in range(2)]
    torch.cuda.synchronize()
    call(x, r, *got, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    held = [torch.zeros_like(x), torch.zeros_like(x)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*held, *got)
    for a, b in ((x, r), (r, x), (x, r)):
        held[0].copy_(a)
        held[1].copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        call(a, b, *want)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_no_rows():
    log("[test] post_norm no rows")
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    _lib.moe_w4a4_post_norm(e, e, e, EPS)
    torch.cuda.synchronize()


@pytest.mark.parametrize("cols", [512, 2048, 4096, 16384, 32768])
@pytest.mark.parametrize("res_f32", [False, True])
def test_infinity_in_a_row(cols, res_f32):
    """x / sqrt(mean x^2) with an infinity in the row: 0 for the finite values, whose stream
    stays as it is, and NaN in its own place; an infinity in the stream does the same to y.
    Exact: nothing is rounded."""
    log(f"[test] post norm of rows with an infinity, cols {cols} float32 stream {res_f32}")
    rng = np.random.default_rng(cols)
    xd, rd = typed(rng.normal(size=(4, cols)), False)[0], typed(rng.normal(size=(4, cols)), res_f32)[0]
    xd[1, 5], xd[2, cols - 1] = float("inf"), float("-inf")
    w = torch.ones(cols, device="cuda")
    at = torch.zeros((4, cols), dtype=torch.bool, device="cuda")
    at[1, 5] = at[2, cols - 1] = True
    ro = torch.empty_like(rd)
    _lib.moe_w4a4_post_norm(xd, rd, ro, EPS, post_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(ro), at)
    assert torch.equal(ro[1:3][~at[1:3]], rd[1:3][~at[1:3]])
    y = torch.empty_like(xd)
    _lib.moe_w4a4_post_norm(xd, rd, ro, EPS, next_weight=w, y=y)
    torch.cuda.synchronize()
    assert torch.equal(ro[at], xd[at].to(ro.dtype)) and not torch.any(torch.isinf(ro[~at]))
    assert torch.equal(torch.isnan(y), at) and torch.all(y[1:3][~at[1:3]] == 0) and torch.all(torch.isfinite(y[::3]))


# ---- the block that ends with it ---------------------------------------------------
H, I, E, K = 512, 256, 16, 3
ROUTE = dict(scoring=_lib.MOE_SCORE_SQRTSOFTPLUS, num_groups=4, topk_groups=2, renormalize=True, scale=1.5)


def bf(rng, *shape, scale=1.0):
    return dev_bf16(bf16.encode((scale * rng.normal(size=shape)).astype(np.float32).astype(np.float64)))


def block(kind, T):
    rng = np.random.default_rng(3)
    gate = Bf16Linear(bf(rng, E, H, scale=0.05))
    mlp = Bf16MLP(Bf16Linear(bf(rng, 2 * I, H, scale=0.04), function=_lib.MOE_FN_SILU, gated=True),
                  Bf16Linear(bf(rng, H, I, scale=0.06)))
    if kind == "bf16":
        return Bf16Experts(bf(rng, E, 2 * I, H, scale=0.04), bf(rng, E, H, I, scale=0.06), K, T), gate, mlp
    layer = layer_for(H, I, E, K, T, mma_type=MX4)
    layer.load_fp32(lambda e: synth.expert_weights_f32(synth.LayerConfig(160, "b", T, H, I, E, K, "uniform", 160), e), threads=4)
    return layer, gate, mlp


@pytest.mark.parametrize("kind", ["w4a4", "bf16"])
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
def test_block_equals_its_steps(kind, res):
    """Norm, a bfloat16 gate's float32 logits, router, experts, a shared MLP and the norm behind
    them: the bits of the steps called one by one; two blocks in a row share the stream."""
    log(f"[test] block {kind} residual {res} with a shared MLP and a norm behind")
    T = 2800
    layer, gate, mlp = block(kind, T)
    rng = np.random.default_rng(4)
    x, r = bf(rng, T, H), bf(rng, T, H, scale=2.0)
    w, b = torch.ones(H, device="cuda"), dev((0.1 * rng.normal(size=E)).astype(np.float32))
    pw, nw, pg = (dev((1 + 0.1 * rng.normal(size=H)).astype(np.float32)) for _ in range(3))
    r = None if res is None else r.float() * 1.001 if res == "f32" else r
    for n in (0, 1, 40, T):
        rn = None if r is None else r[:n].clone()
        kept = x[:n].clone()
        y2, h2 = layer.forward_block(x[:n], rn, w, EPS, gate, bias=b, shared=mlp, post_weight=pw, post_gate=pg, post_scale=0.5,
                                     next_weight=nw, **ROUTE)
        y, ro = torch.empty_like(x[:n]), None if r is None else torch.empty_like(rn)
        _lib.moe_w4a4_add_rmsnorm(x[:n], rn, w, EPS, residual_out=ro, y=y)
        h = x[:n] if r is None else ro
        logits = torch.empty((n, E), device="cuda")
        _lib.moe_w4a4_linear_bf16(y, gate.weight, logits)
        ids, rw = torch.empty((n, K), dtype=torch.int32, device="cuda"), torch.empty((n, K), device="cuda")
        _lib.moe_w4a4_router(logits, ids, rw, bias=b, **ROUTE)
        out = layer.forward(y, ids, rw)
        out = mlp.forward(y, addend=out)
        want_h, want_y = torch.empty_like(h), torch.empty_like(out)
        _lib.moe_w4a4_post_norm(out, h, want_h, EPS, post_weight=pw, gate=pg, scale=0.5, next_weight=nw, y=want_y)
        torch.cuda.synchronize()
        assert torch.equal(y2, want_y) and torch.equal(h2, want_h) and torch.equal(x[:n], kept)
        if r is not None:
            assert torch.equal(rn, r[:n])
        none, h3 = layer.forward_block(x[:n], rn, w, EPS, gate, bias=b, shared=mlp, post_weight=pw, post_gate=pg, post_scale=0.5,
                                       **ROUTE)
        torch.cuda.synchronize()
        assert none is None and torch.equal(h3, want_h)


@pytest.mark.parametrize("kind", ["w4a4", "bf16"])
def test_block_without_a_norm_behind_and_on_another_stream(kind):
    log(f"[test] block {kind}: plain return, stream argument")
    T = 40
    layer, gate, mlp = block(kind, T)
    rng = np.random.default_rng(5)
    x, r, w = bf(rng, T, H), bf(rng, T, H), torch.ones(H, device="cuda")
    out, h = layer.forward_block(x, r, w, EPS, gate, shared=mlp, **ROUTE)
    y2, h2 = layer.forward_block(x, r, w, EPS, gate, shared=mlp, post_scale=0.3, next_weight=w, **ROUTE)
    want_h, want_y = torch.empty_like(h), torch.empty_like(out)
    _lib.moe_w4a4_post_norm(out, h, want_h, EPS, scale=0.3, next_weight=w, y=want_y)
    torch.cuda.synchronize()
    assert torch.equal(y2, want_y) and torch.equal(h2, want_h)
    side = torch.cuda.Stream()
    r2 = r.clone()
    torch.cuda.synchronize()
    y3, h3 = layer.forward_block(x, r2, w, EPS, gate, residual_out=r2, shared=mlp, post_scale=0.3, next_weight=w,
                                 stream=side.cuda_stream, **ROUTE)
    side.synchronize()
    assert h3 is r2 and torch.equal(y3, want_y) and torch.equal(r2, want_h)


@pytest.mark.parametrize("T", [1, 300])
def test_block_of_bf16_experts_captured(T):
    log(f"[test] block bf16 T {T} in a graph")
    layer, gate, mlp = block("bf16", T)
    w = torch.ones(H, device="cuda")
    sets = [[bf(np.random.default_rng(s), T, H), bf(np.random.default_rng(s + 10), T, H)] for s in (6, 7)]

    def call(a, out=None, h=None):
        return layer.forward_block(a[0], a[1], w, EPS, gate, residual_out=h, shared=mlp, out=out, post_weight=w, next_weight=w,
                                   **ROUTE)

    eager = [[t.clone() for t in call(a)] for a in sets]
    held = [t.clone() for t in sets[0]]
    out, h = torch.empty_like(held[0]), torch.empty_like(held[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(held, out, h)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(held, out, h)
    for which in (1, 0, 1):
        for dst, src in zip(held, sets[which]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[which][0]) and torch.equal(h, eager[which][1])
        other = call(sets[1 - which])
        torch.cuda.synchronize()
        assert torch.equal(other[0], eager[1 - which][0])
