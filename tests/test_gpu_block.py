"""GPU tier: the operators around the layer together, as a decoder block uses
them (MoeW4A4Layer.forward_block): residual addition and norm, router logits,
the router's choice, the routed experts and a shared linear -- against the fp64
oracles run on the device's own inputs of each step, on another stream, and
captured into a graph.

Tolerances are those of the operators' own tests: h and y exact but next to a
border, ids equal, weights 2^-18, the experts' output the layer's parity bar
(relative 2-norm 5e-3), the shared linear oracle.linear.sum_error and half a step
of bfloat16."""
import numpy as np
import pytest
import torch

import synth
from block_scaled_fp4_pre_amd import _lib
from block_scaled_fp4_pre_amd.layer import W4A4Linear
from oracle import bf16, linear, mxfp4, norm, router
from oracle.forward import forward
from tests.gpu_support import dev, dev_bf16, host_bits, layer_for, log
from tests.oracle_inputs import all_expert_weights

pytestmark = pytest.mark.gpu

H, I, E, K = 512, 256, 16, 3
MX4, FP8 = _lib.MOE_MMA_MXF4_X_MXF4, _lib.MOE_MMA_FP8_X_MXF4


def config(T):
    return synth.LayerConfig(160, "block_h512_i256_e16_k3", T, H, I, E, K, "uniform", 160)


def block(T, mma):
    layer = layer_for(H, I, E, K, T, mma_type=mma)
    layer.load_fp32(lambda e: synth.expert_weights_f32(config(T), e), threads=4)
    rng = np.random.default_rng(1)
    wc, ws = mxfp4.quantize_packed((0.02 * rng.normal(size=(H, H))).astype(np.float32))
    shared = W4A4Linear(H, H, T, mma_type=mma)
    shared.load_canonical(dev(wc), dev(ws))
    gate = bf16.encode((0.05 * rng.normal(size=(E, H))).astype(np.float32).astype(np.float64))
    return layer, shared, (wc, ws), gate


def inputs(T, seed):
    rng = np.random.default_rng(seed)
    enc = lambda v: bf16.encode(v.astype(np.float32).astype(np.float64))  # noqa: E731
    return (enc(rng.normal(size=(T, H))), enc(2 * rng.normal(size=(T, H))),
            (1 + 0.1 * rng.normal(size=H)).astype(np.float32), (0.1 * rng.normal(size=E)).astype(np.float32))


ROUTE = dict(scoring=_lib.MOE_SCORE_SQRTSOFTPLUS, num_groups=4, topk_groups=2, renormalize=True, scale=1.5)


@pytest.mark.parametrize("mma,name", [(MX4, "mxf4xmxf4"), (FP8, "fp8xfp4")])
@pytest.mark.parametrize("T", [1, 16, 100, 2800])       # 2800: 8400 routed rows, the norm quantizes
def test_block_against_the_oracles(T, mma, name):
    log(f"[test] block T {T} {name}")
    layer, shared, (wc, ws), gate = block(T, mma)
    x, r, w, b = inputs(T, T)
    gd = dev_bf16(gate)
    out, h = layer.forward_block(dev_bf16(x), dev_bf16(r), dev(w), 1e-6, gd, bias=dev(b), shared=shared, **ROUTE)
    torch.cuda.synchronize()
    hv = norm.residual_sum(bf16.decode(x), bf16.decode(r), True)
    assert np.array_equal(host_bits(h), bf16.encode(hv))
    y = norm.round_y(norm.rmsnorm(hv, w, 1e-6))
    # the logits as the library's product gives them on this y (its own rounding)
    logits = torch.nn.functional.linear(dev_bf16(y), gd).float().cpu().numpy()
    sub = np.arange(T) if T <= 100 else np.random.default_rng(2).choice(T, 60, replace=False)
    ids, rw = router.route_logits(logits, K, "sqrtsoftplus", b, 4, 2, True, 1.5)
    ref = forward(y[sub], ids[sub], rw[sub].astype(np.float32), all_expert_weights(config(T)), E, I,
                  mma_type=name)["out_f64"]
    # without the shared linear first
    alone, _ = layer.forward_block(dev_bf16(x), dev_bf16(r), dev(w), 1e-6, gd, bias=dev(b), **ROUTE)
    torch.cuda.synchronize()
    got = bf16.decode(host_bits(alone))
    assert np.linalg.norm(got[sub] - ref) / np.linalg.norm(ref) <= 5e-3
    c, s = linear.quantize_tokens(bf16.decode(y), mma == FP8)
    full, mag = linear.linear(c, s, wc, ws, mma == FP8, got)
    tol = linear.sum_error(mag + np.abs(got), H, mma == FP8)
    tol = tol + (np.abs(full) + tol) * 2.0 ** -8
    assert np.all(np.abs(bf16.decode(host_bits(out)) - full) <= tol)


@pytest.mark.parametrize("T", [5, 2800])
def test_block_on_another_stream_and_with_a_w4a4_gate(T):
    log(f"[test] block T {T}: stream argument, W4A4 gate, in-place residual")
    layer, shared, _, gate = block(T, MX4)
    g = W4A4Linear(H, E, T)
    g.load_fp32(torch.from_numpy(bf16.decode(gate).astype(np.float32)))
    x, r, w, b = (dev_bf16(v) if v.dtype == np.uint16 else dev(v) for v in inputs(T, 3))
    first = layer.forward_block(x, r, w, 1e-6, g, bias=b, shared=shared, **ROUTE)
    torch.cuda.synchronize()
    side, r2, out = torch.cuda.Stream(), r.clone(), torch.empty_like(first[0])
    torch.cuda.synchronize()
    got = layer.forward_block(x, r2, w, 1e-6, g, residual_out=r2, bias=b, shared=shared, out=out,
                              stream=side.cuda_stream, **ROUTE)
    side.synchronize()
    assert torch.equal(got[0], first[0]) and torch.equal(r2, first[1])
    with pytest.raises(ValueError):
        layer.forward_block(torch.cat([x, x]), torch.cat([r, r]), w, 1e-6, g)


@pytest.mark.parametrize("T", [1, 40, 600, 2800])
def test_block_captured_and_replayed(T):
    """Replayed three times on new inputs with eager calls on the same
    workspaces in between; every replay equals the eager call bit for bit."""
    log(f"[test] block T {T} in a graph")
    layer, shared, _, gate = block(T, FP8)
    gw = dev_bf16(gate)
    sets = [[dev_bf16(v) if v.dtype == np.uint16 else dev(v) for v in inputs(T, s)] for s in (4, 5)]

    def call(a, out=None, h=None):
        x, r, w, b = a
        return layer.forward_block(x, r, w, 1e-6, gw, residual_out=h, bias=b, shared=shared, out=out, **ROUTE)

    eager = [call(a) for a in sets]
    torch.cuda.synchronize()
    held = [t.clone() for t in sets[0]]
    out, h = torch.empty_like(eager[0][0]), torch.empty_like(eager[0][1])
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


def test_linears_on_two_streams_with_their_own_workspaces():
    log("[test] two linears at once")
    rng = np.random.default_rng(6)
    wc, ws = mxfp4.quantize_packed((0.02 * rng.normal(size=(1024, 1024))).astype(np.float32))
    base = W4A4Linear(1024, 1024, 300)
    base.load_canonical(dev(wc), dev(ws))
    lins = [base, base.with_capacity(300)]
    xs = [dev_bf16(inputs(600, s)[0].reshape(300, 1024)) for s in (7, 8)]
    want = [l.forward(x) for l, x in zip(lins, xs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    for i in range(20):
        for l, x, s, o in zip(lins, xs, streams, outs):
            l.forward(x, out=o[i], stream=s.cuda_stream)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, t) for t in o)


def on_another_stream(call):
    """call(stream) -> new output tensors, filled on another stream while the
    current one still has to read memory that was freed after it: the outputs
    must not lie there."""
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    held = [torch.full_like(t, 3.0) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                     # the current stream is busy for a while
    kept = [t.clone() for t in held]
    places = [t.data_ptr() for t in held]
    del held
    got = call(side.cuda_stream)
    assert not {t.data_ptr() for t in got} & set(places)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 3.0).all()) for t in kept)


@pytest.mark.parametrize("T", [5, 300])
def test_new_outputs_are_of_the_streams_own_memory(T):
    log(f"[test] T {T}: outputs made for another stream")
    layer, shared, _, gate = block(T, MX4)
    x, r, w, b = (dev_bf16(v) if v.dtype == np.uint16 else dev(v) for v in inputs(T, 9))
    gd = dev_bf16(gate)
    ids = torch.arange(T * K, dtype=torch.int32, device="cuda").view(T, K) % E
    rw = torch.full((T, K), 0.5, device="cuda")
    on_another_stream(lambda s: [shared.forward(x, stream=s)])
    on_another_stream(lambda s: [shared.forward(x, dtype=torch.float32, stream=s)])
    on_another_stream(lambda s: [layer.forward(x, ids, rw, stream=s)])
    on_another_stream(lambda s: list(layer.forward_block(x, r, w, 1e-6, gd, bias=b, shared=shared, stream=s, **ROUTE)))


@pytest.mark.parametrize("T", [5, 2800])
def test_handle_of_the_default_stream(T):
    """stream=0, which is what torch's default stream has for a handle: the call
    follows what that stream still has to do."""
    log(f"[test] block T {T} on the default stream by its handle")
    layer, shared, _, gate = block(T, MX4)
    x, r, w, b = (dev_bf16(v) if v.dtype == np.uint16 else dev(v) for v in inputs(T, 10))
    gd, late = dev_bf16(gate), torch.zeros_like(x)
    assert torch.cuda.current_stream().cuda_stream == 0
    want = layer.forward_block(x, r, w, 1e-6, gd, bias=b, shared=shared, **ROUTE)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    late.copy_(x)
    got = layer.forward_block(late, r, w, 1e-6, gd, bias=b, shared=shared, stream=0, **ROUTE)
    lin = shared.forward(late, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(lin, shared.forward(x))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                # also where another stream is the current one
        again = layer.forward_block(late, r, w, 1e-6, gd, bias=b, shared=shared, stream=0, **ROUTE)
    torch.cuda.synchronize()
    assert torch.equal(again[0], want[0])


@pytest.mark.parametrize("mma", [MX4, FP8, _lib.MOE_MMA_NVF4_X_NVF4], ids=["mxf4xmxf4", "fp8xfp4", "nvf4xnvf4"])
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
def test_block_equals_its_steps(mma, res):
    """Every type and residual, no tokens among the counts: the bits of the
    steps called one by one."""
    log(f"[test] block type {mma} residual {res}")
    T = 2800
    if mma == _lib.MOE_MMA_NVF4_X_NVF4:
        layer = layer_for(H, I, E, K, T, mma_type=mma)
        scales = np.full(E, 2.0 ** -14, np.float32)
        layer.load_fp32(lambda e: synth.expert_weights_f32(config(T), e), threads=4,
                        tensor_scales=(2.0 ** -8, 2.0 ** -8, scales, scales))
        shared = block(T, MX4)[1]
        gate = block(T, MX4)[3]
    else:
        layer, shared, _, gate = block(T, mma)
    x, r, w, b = (dev_bf16(v) if v.dtype == np.uint16 else dev(v) for v in inputs(T, 12))
    gd = dev_bf16(gate).t().contiguous().t()              # a gate stored the other way round
    r = None if res is None else r.float() * 1.001 if res == "f32" else r
    for n in (0, 1, 40, T):
        rn = None if r is None else r[:n].clone()
        out, h = layer.forward_block(x[:n], rn, w, 1e-6, gd, bias=b, shared=shared, **ROUTE)
        y, ro = torch.empty_like(x[:n]), None if r is None else torch.empty_like(rn)
        _lib.moe_w4a4_add_rmsnorm(x[:n], rn, w, 1e-6, residual_out=ro, y=y)
        ids, rw = torch.empty((n, K), dtype=torch.int32, device="cuda"), torch.empty((n, K), device="cuda")
        _lib.moe_w4a4_router(torch.nn.functional.linear(y, gd), ids, rw, bias=b, **ROUTE)
        want = shared.forward(y, addend=layer.forward(y, ids, rw))
        torch.cuda.synchronize()
        assert out.shape == (n, H) and torch.equal(out, want)
        assert h is x[:n] or torch.equal(h, x[:n] if r is None else ro)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_block_under_autocast(dtype):
    """torch's own product of the gate keeps its type, whatever autocast asks for."""
    log(f"[test] block under autocast to {dtype}")
    layer, shared, _, gate = block(40, MX4)
    x, r, w, b = (dev_bf16(v) if v.dtype == np.uint16 else dev(v) for v in inputs(40, 13))
    gd = dev_bf16(gate)
    want = layer.forward_block(x, r, w, 1e-6, gd, bias=b, shared=shared, **ROUTE)
    r2 = r.clone()
    with torch.autocast("cuda", dtype=dtype):
        got = layer.forward_block(x, r2, w, 1e-6, gd, residual_out=r2, bias=b, shared=shared, **ROUTE)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(r2, want[1])
