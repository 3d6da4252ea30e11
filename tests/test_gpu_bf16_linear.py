"""GPU tier: moe_w4a4_linear_bf16, moe_w4a4_grouped_linear_bf16 and moe_w4a4_experts_bf16 against
the fp64 oracle.

Tolerance: the bound of oracle.bf16_linear.linear on a device's sums, then half a step of the
output's type: 2^-8 (bfloat16), 2^-24 (float32) of the value.  The experts' h and y are each
rounded to bfloat16 and may fall on the other side of a border: the layer's parity
bar (relative 2-norm 5e-3), and bit for bit the steps called one by one."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from block_scaled_fp4_pre_amd.layer import Bf16Experts, Bf16Linear, Bf16MLP
from oracle import bf16, bf16_linear
from oracle.route import route
from tests.gpu_support import dev, dev_bf16, host_bits, log

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
FN = {name: i for i, name in enumerate(bf16_linear.FUNCTIONS)}


def rounded(v):
    """(bits, fp64 values) of v in bfloat16."""
    bits = bf16.encode(np.asarray(v, np.float32).astype(np.float64))
    return bits, bf16.decode(bits)


def rows_like(rng, T, K):
    return rounded(rng.normal(size=(T, K)) * np.exp(0.5 * rng.normal(size=K)) * np.exp(0.3 * rng.normal(size=(T, 1))))


def weights(rng, *shape):
    return rounded(rng.normal(size=shape) / np.sqrt(shape[-1]))


def values(t):
    return t.double().cpu().numpy() if t.dtype is F32 else bf16.decode(host_bits(t))


def close(got, ref, bound, f32):
    tol = bound + (np.abs(ref) + bound) * (2.0 ** -24 if f32 else 2.0 ** -8)
    err = np.abs(got - ref)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(~(err <= tol))[:4])


def typed(rng, shape, f32, scale=1.0):
    """A device tensor of either type and its values."""
    v = (scale * rng.normal(size=shape)).astype(np.float32)
    if f32:
        return dev(v), v.astype(np.float64)
    bits, v = rounded(v)
    return dev_bf16(bits), v


def strided(t, pad, fill):
    """t as the first columns of rows that are `pad` wider, the rest `fill`."""
    wide = torch.full((t.shape[0] + 2, t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    wide[:t.shape[0], :t.shape[1]] = t
    return wide, wide[:t.shape[0], :t.shape[1]]


def run_linear(T, K, N, fn="none", gated=False, bias=None, scale=False, add=None, f32=False, pad=0, seed=0):
    """bias, add: None, False (bfloat16) or True (float32)."""
    rng = np.random.default_rng([T, K, N, seed])
    xb, x = rows_like(rng, T, K)
    wb, w = weights(rng, 2 * N if gated else N, K)
    bd = b = ad = a = sd = s = None
    if bias is not None:
        bd, b = typed(rng, w.shape[0], bias, 0.3)
    if add is not None:
        ad, a = typed(rng, (T, N), add)
        if pad:
            ad = strided(ad, 5, 0)[1]
    if scale:
        sd, s = typed(rng, T, True)
    xd = dev_bf16(xb)
    if pad:
        xd = strided(xd, pad, float("nan"))[1]          # (what lies between the rows is not read)
    out_wide, out = strided(torch.zeros((T, N), dtype=F32 if f32 else BF, device="cuda"), 3 if pad else 0, 77.0)
    _lib.moe_w4a4_linear_bf16(xd, dev_bf16(wb), out, bias=bd, function=FN[fn], gated=gated, row_scale=sd, addend=ad)
    torch.cuda.synchronize()
    assert torch.all(out_wide[T:] == 77.0) and torch.all(out_wide[:, N:] == 77.0)
    ref, bound = bf16_linear.linear(x, w, fn, gated, b, s, a)
    close(values(out), ref, bound, f32)


SIZES = [(1, 8, 1), (1, 64, 16), (1, 4096, 256), (1, 1000, 77), (2, 96, 17), (3, 128, 64), (7, 4096, 512), (8, 72, 100),
         (15, 2048, 65), (16, 2080, 256), (16, 65536, 8), (17, 1056, 257), (31, 4096, 130), (32, 512, 1111), (33, 8192, 48),
         (48, 96, 2048), (63, 1024, 63), (64, 2048, 512), (65, 256, 300), (100, 1600, 1023), (128, 128, 128), (130, 416, 515),
         (129, 8, 129), (193, 56, 33), (255, 2048, 255), (256, 1024, 1024), (257, 64, 2048), (300, 1064, 1111), (513, 640, 260),
         (1030, 4096, 256), (1000, 8, 3), (2050, 72, 4100), (4097, 136, 640)]


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_sizes(T, K, N, gated):
    log(f"[test] linear_bf16 T {T} K {K} N {N} gated {gated}")
    run_linear(T, K, N, fn="silu" if gated else "none", gated=gated)


# one size for each kernel: a few rows, 32, 64, tiles of 128 and of 256
FORMS = [(5, 200, 37), (29, 264, 50), (50, 456, 70), (150, 328, 141), (1100, 72, 4200)]


@pytest.mark.parametrize("T,K,N", FORMS)
@pytest.mark.parametrize("fn", bf16_linear.FUNCTIONS)
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_functions_with_everything_in_the_epilogue(T, K, N, fn, gated):
    log(f"[test] linear_bf16 T {T} K {K} N {N} {fn} gated {gated}, epilogue")
    run_linear(T, K, N, fn, gated, bias=True, scale=True, add=False, seed=1)
    run_linear(T, K, N, fn, gated, bias=False, scale=True, add=True, f32=True, pad=8, seed=2)


@pytest.mark.parametrize("T,K,N", FORMS)
@pytest.mark.parametrize("bias,scale,add,f32,pad", [(None, False, None, True, 0), (True, False, None, False, 0),
                                                    (None, True, None, False, 72), (None, False, True, False, 0),
                                                    (None, False, False, True, 8), (False, False, None, True, 0)])
def test_types_and_strides(T, K, N, bias, scale, add, f32, pad):
    log(f"[test] linear_bf16 T {T} K {K} N {N} bias {bias} scale {scale} addend {add} f32 {f32} pad {pad}")
    run_linear(T, K, N, bias=bias, scale=scale, add=add, f32=f32, pad=pad, seed=3)


@pytest.mark.parametrize("T,K,N", FORMS)
@pytest.mark.parametrize("f32", [False, True])
def test_addend_in_the_place_of_out(T, K, N, f32):
    log(f"[test] linear_bf16 T {T}: in place, f32 {f32}")
    rng = np.random.default_rng(4)
    lin = Bf16Linear(dev_bf16(weights(rng, N, K)[0]))
    x = dev_bf16(rows_like(rng, T, K)[0])
    out = typed(rng, (T, N), f32)[0]
    want = lin.forward(x, addend=out, dtype=out.dtype)
    assert lin.forward(x, out=out, addend=out) is out
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T,K,N", FORMS)
def test_non_finite_rows_stay_alone(T, K, N):
    """A row with infinities and NaN, weights of a padded tile's neighbours, and the piece
    behind K of a sliced row: each stays where it is."""
    log(f"[test] linear_bf16 T {T}: non-finite row")
    rng = np.random.default_rng(5)
    wb, w = weights(rng, N, K)
    xb, x = rows_like(rng, T, K)
    bad = xb.copy()
    bad[T - 1, 0] = 0x7F80                                   # in the first piece
    bad[T - 1, K - 1] = 0x7FC0 if T % 2 else 0x7F80          # in the last one
    w0 = wb.copy()
    w0[N - 1, :] = 0x7F80
    clean = torch.empty((T, N), device="cuda")
    got = torch.empty((T, N), device="cuda")
    _lib.moe_w4a4_linear_bf16(dev_bf16(xb), dev_bf16(wb), clean)
    wide = torch.full((T, K + 8), float("nan"), dtype=BF, device="cuda")
    wide[:, :K] = dev_bf16(bad)
    _lib.moe_w4a4_linear_bf16(wide[:, :K], dev_bf16(w0), got)
    torch.cuda.synchronize()
    assert torch.equal(got[:T - 1, :N - 1], clean[:T - 1, :N - 1])
    assert not torch.isfinite(got[T - 1]).any() and not torch.isfinite(got[:, N - 1]).any()


@pytest.mark.parametrize("fn", ["silu", "gelu", "gelu_tanh"])
def test_functions_over_their_whole_range(fn):
    """One term a sum, so that f's argument is exact: every exponent, tails and borders."""
    log(f"[test] linear_bf16 {fn} over its range")
    v = np.concatenate([np.linspace(-110, 110, 4001), 2.0 ** np.arange(-140, 100, 3), -(2.0 ** np.arange(-140, 100, 3)), [0.0]])
    bits, v = rounded(v)
    x = np.zeros((len(v), 8), np.uint16)
    x[:, 0] = bits
    w = np.zeros((4, 8), np.uint16)
    w[:, 0] = 0x3F80
    out = torch.empty((len(v), 4), device="cuda")
    _lib.moe_w4a4_linear_bf16(dev_bf16(x), dev_bf16(w), out, function=FN[fn])
    torch.cuda.synchronize()
    ref = bf16_linear.apply(fn, v)
    err = np.abs(out.cpu().numpy().astype(np.float64) - ref[:, None])
    tol = np.abs(ref) * (2.0 ** -20 + 2.0 ** -24) + 2.0 ** -126
    assert np.all(err <= tol[:, None]), (float((err / tol[:, None]).max()), v[np.argmax((err / tol[:, None]).max(1))])


def test_deterministic_and_on_another_stream():
    log("[test] linear_bf16 twice, on a stream of its own, and by the default stream's handle")
    rng = np.random.default_rng(6)
    for T, K, N in FORMS:
        lin = Bf16Linear(dev_bf16(weights(rng, 2 * N, K)[0]), function=FN["silu"], gated=True)
        x = dev_bf16(rows_like(rng, T, K)[0])
        want = lin.forward(x)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = lin.forward(x, stream=side.cuda_stream)
        side.synchronize()
        torch.cuda._sleep(50_000_000)
        late = torch.zeros_like(x)
        late.copy_(x)
        zero = lin.forward(late, stream=0)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(zero, want) and torch.equal(lin.forward(x), want)


def test_no_tokens():
    log("[test] linear_bf16 no tokens")
    lin = Bf16Linear(torch.zeros((32, 64), dtype=BF, device="cuda"))
    assert lin.forward(torch.empty((0, 64), dtype=BF, device="cuda")).shape == (0, 32)
    w = torch.zeros((3, 32, 64), dtype=BF, device="cuda")
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    _lib.moe_w4a4_grouped_linear_bf16(torch.empty((0, 64), dtype=BF, device="cuda"), w, offsets,
                                      torch.empty((0, 32), dtype=BF, device="cuda"))
    torch.cuda.synchronize()


def test_rows_past_32_bit_offsets():
    """Outputs and inputs of more than 2^31 elements and 2^32 bytes: the first, the last and
    some rows between them."""
    log("[test] linear_bf16 far rows")
    T, K, N, wide = 530000, 8, 24, 4096
    x = torch.zeros((T, wide), dtype=BF, device="cuda")
    out = torch.zeros((T, 4200), dtype=BF, device="cuda")
    rng = np.random.default_rng(7)
    wb, w = weights(rng, N, K)
    at = [0, 1, 262143, 262144, 524287, 524288, T - 1]
    xb, xv = rows_like(rng, len(at), K)
    x[at, :K] = dev_bf16(xb)
    _lib.moe_w4a4_linear_bf16(x[:, :K], dev_bf16(wb), out[:, :N])
    torch.cuda.synchronize()
    close(values(out[at][:, :N].contiguous()), *bf16_linear.linear(xv, w), False)
    assert int((out != 0).any(1).sum()) == len(at) and not bool((out[:, N:] != 0).any())


# ---- grouped ---------------------------------------------------------------------
def run_grouped(counts, K, N, fn="none", gated=False, divisor=0, bias=None, scale=False, add=None, f32=False, before=0,
                behind=0, seed=0):
    """Groups of `counts` rows, `before` rows ahead of them and `behind` behind."""
    rng = np.random.default_rng([len(counts), sum(counts), K, N, seed])
    E, R = len(counts), before + sum(counts) + behind
    offsets = before + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = None
    Tx = R
    if divisor:
        Tx = max(1, -(-sum(counts) // divisor))
        rows = rng.integers(0, Tx * divisor, size=R).astype(np.int32)
    xb, x = rows_like(rng, Tx, K)
    wb, w = weights(rng, E, 2 * N if gated else N, K)
    bd = b = sd = s = ad = a = None
    if bias is not None:
        bd, b = typed(rng, w.shape[:2], bias, 0.3)
    if scale:
        sd, s = typed(rng, R, True)
    if add is not None:
        ad, a = typed(rng, (R, N), add)
    out = torch.full((R + 1, N), 77.0, dtype=F32 if f32 else BF, device="cuda")
    _lib.moe_w4a4_grouped_linear_bf16(dev_bf16(xb), dev_bf16(wb), dev(offsets), out[:R], rows=None if rows is None else dev(rows),
                                      row_divisor=max(1, divisor), bias=bd, function=FN[fn], gated=gated, row_scale=sd, addend=ad)
    torch.cuda.synchronize()
    ref, bound = bf16_linear.grouped(x, w, offsets, rows, max(1, divisor), fn, gated, b, s, a)
    ref = ref if rows is not None or Tx == R else ref[:R]
    a0, b0 = offsets[0], offsets[-1]
    assert torch.all(out[:a0] == 77.0) and torch.all(out[b0:] == 77.0)
    close(values(out[a0:b0]), ref[a0:b0], bound[a0:b0], f32)


COUNTS = {
    "one": [1], "one_of_many": [0] * 40 + [1] + [0] * 23, "few": [1, 0, 2, 1, 0, 0, 1, 3], "sixteens": [16, 15, 17, 0, 32, 33],
    "hot": [200, 1, 0, 3, 1, 1], "thirty": [30, 20, 31, 0, 25, 33], "sixty": [64, 40, 65, 50, 61, 0, 63], "tiles": [128, 129, 0, 127, 300, 1],
    "wide": [256, 257, 700, 0, 1, 255], "e512": [int(c) for c in np.random.default_rng(0).integers(0, 4, 512)], "none": [0, 0, 0],
    "big": [600, 900, 0, 511, 513, 1024, 3],
}


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("K,N", [(136, 33), (200, 260), (64, 512)])
def test_groups(name, gated, K, N):
    log(f"[test] grouped_bf16 {name} K {K} N {N} gated {gated}")
    if name == "e512" and N > 260:
        K, N = 64, 40
    run_grouped(COUNTS[name], K, N, "silu" if gated else "none", gated, divisor=0, before=2, behind=3)
    run_grouped(COUNTS[name], K, N, "gelu" if gated else "none", gated, divisor=3, seed=1)


@pytest.mark.parametrize("name", ["few", "thirty", "sixty", "tiles", "big"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_groups_with_everything_in_the_epilogue(name, gated):
    log(f"[test] grouped_bf16 {name} epilogue gated {gated}")
    run_grouped(COUNTS[name], 72, 45, "gelu_tanh", gated, 2, True, True, False, before=1, behind=2)
    run_grouped(COUNTS[name], 328, 130, "silu", gated, 0, False, True, True, f32=True, behind=5)


@pytest.mark.parametrize("R,N", [(40, 33), (400, 200), (3000, 64)])
def test_wrong_offsets_and_rows_stay_inside(R, N):
    """Offsets and rows that the host cannot read: whatever they hold, nothing outside the
    tensors is written (and the call ends)."""
    log(f"[test] grouped_bf16 wrong offsets, {R} rows")
    K, E = 64, 5
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randn((E, N, K), generator=g, device="cuda").to(BF)
    x = torch.randn((7, K), generator=g, device="cuda").to(BF)
    rows = torch.randint(-2 ** 31, 2 ** 31 - 1, (R,), generator=g, device="cuda", dtype=torch.int32)
    for bad in ([0, 10, 5, R + 1000, -7, R], [2 ** 31 - 1, -2 ** 31, 0, R, R, 3], [-5, -4, -3, -2, -1, 0], [R, R, R, R, R, R + 1]):
        buf = torch.full((R + 8, N), 77.0, dtype=BF, device="cuda")
        _lib.moe_w4a4_grouped_linear_bf16(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), buf[4:4 + R], rows=rows)
        torch.cuda.synchronize()
        assert torch.all(buf[:4] == 77.0) and torch.all(buf[4 + R:] == 77.0)


# ---- weights past what the caches keep ---------------------------------------------
def device_product(x, w, gated):
    """(fp64 values, bound) of x W^T (gated: SwiGLU) by torch's fp64 products on the device;
    the bound as oracle.bf16_linear.linear's."""
    x, w = x.double(), w.double()
    v, err = x @ w.t().contiguous(), (x.shape[1] + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t().contiguous())
    if not gated:
        return v, err + 2.0 ** -126
    n = v.shape[1] // 2
    f = v[:, :n] * torch.sigmoid(v[:, :n])
    e = 1.11 * err[:, :n] + f.abs() * 2.0 ** -20 + 2.0 ** -126
    out = f * v[:, n:]
    return out, v[:, n:].abs() * e + f.abs() * err[:, n:] + e * err[:, n:] + out.abs() * 2.0 ** -23 + 2.0 ** -126


def device_close(got, ref, bound):
    err, tol = (got.double() - ref).abs(), bound + (ref.abs() + bound) * 2.0 ** -8
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("T", [1, 3, 8, 9, 16, 17, 32, 33, 100])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_many_weights(T, gated):
    log(f"[test] linear_bf16 many weights, T {T} gated {gated}")
    g = torch.Generator(device="cuda").manual_seed(T)
    K, N = 4168, 8201 if gated else 16401
    x = torch.randn((T, K), generator=g, device="cuda").to(BF)
    w = (torch.randn((2 * N if gated else N, K), generator=g, device="cuda") / 64).to(BF)
    out = torch.full((T + 1, N), 77.0, dtype=BF, device="cuda")
    _lib.moe_w4a4_linear_bf16(x, w, out[:T], function=FN["silu"] if gated else 0, gated=gated)
    torch.cuda.synchronize()
    assert torch.all(out[T] == 77.0)
    device_close(out[:T], *device_product(x, w, gated))


@pytest.mark.parametrize("mean", [0.3, 1.5, 6, 13, 40, 80, 140, 300])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_many_experts(mean, gated):
    """Every kernel of the groups, by their mean rows; a hot group and empty ones among them."""
    log(f"[test] grouped_bf16 many weights, mean {mean} gated {gated}")
    E, K, N = 48, 1096, 777 if gated else 1411
    rng = np.random.default_rng(int(10 * mean))
    counts = rng.poisson(mean, E)
    counts[5], counts[E - 1] = 0, 0
    counts[7] = int(4 * mean) + 1
    R = int(counts.sum())
    g = torch.Generator(device="cuda").manual_seed(R)
    x = torch.randn((-(-R // 3), K), generator=g, device="cuda").to(BF)
    w = (torch.randn((E, 2 * N if gated else N, K), generator=g, device="cuda") / 33).to(BF)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = torch.randperm(R, generator=g, device="cuda").to(torch.int32)
    out = torch.full((R + 1, N), 77.0, dtype=BF, device="cuda")
    _lib.moe_w4a4_grouped_linear_bf16(x, w, dev(offsets), out[:R], rows=rows, row_divisor=3, function=FN["silu"] if gated else 0,
                                      gated=gated)
    torch.cuda.synchronize()
    assert torch.all(out[R] == 77.0)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            device_close(out[a:b], *device_product(x[(rows[a:b] // 3).long()], w[e], gated))


def test_gathered_rows_past_2_gib():
    """Rows of x more than 2^31 bytes behind its first (which lies as far into its buffer)."""
    log("[test] grouped_bf16 far gathered rows")
    K, N, stride = 64, 40, 4096
    Tx = 500000                                              # 4.1 GB, below 2^31 elements
    buf = torch.zeros((300000 + Tx, stride), dtype=BF, device="cuda")
    x = buf[300000:, :K]
    rng = np.random.default_rng(11)
    at = np.array([0, 1, 262143, 262144, 262145, 400000, Tx - 1], np.int32)
    xb, xv = rows_like(rng, len(at), K)
    x[torch.from_numpy(at.astype(np.int64)).cuda()] = dev_bf16(xb)
    wb, w = weights(rng, 2, N, K)
    out = torch.zeros((len(at), N), dtype=BF, device="cuda")
    _lib.moe_w4a4_grouped_linear_bf16(x, dev_bf16(wb), dev(np.array([0, 3, len(at)], np.int32)), out, rows=dev(at))
    torch.cuda.synchronize()
    for a, b, e in ((0, 3, 0), (3, len(at), 1)):
        close(values(out[a:b]), *bf16_linear.linear(xv[a:b], w[e]), False)


# ---- experts ---------------------------------------------------------------------
def make_experts(rng, H, I, E, k, T):
    (w1b, w1), (w2b, w2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
    return Bf16Experts(dev_bf16(w1b), dev_bf16(w2b), k, T), w1, w2


def routing(rng, T, E, k):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    return ids, rng.random((T, k)).astype(np.float32)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 40, 4, 2), (1, 512, 256, 16, 3), (6, 72, 56, 5, 5), (33, 256, 128, 8, 1),
                                       (100, 136, 200, 12, 4), (700, 64, 72, 3, 2), (1500, 64, 32, 40, 6)])
def test_experts(T, H, I, E, k):
    log(f"[test] experts_bf16 T {T} H {H} I {I} E {E} k {k}")
    rng = np.random.default_rng([T, H])
    layer, w1, w2 = make_experts(rng, H, I, E, k, T)
    layer.workspace.fill_(0xA5)
    xb, x = rows_like(rng, T, H)
    ids, wt = routing(rng, T, E, k)
    ids[0, 0] = -1                                            # a masked slot
    ids[T - 1, 0] = E                                         # and one out of range
    if T > 5:
        ids[3] = -1                                           # a token without experts
        ids[4] = ids[4, 0]                                    # and one with the same expert in every slot
    xd, idd, wd = dev_bf16(xb), dev(ids), dev(wt)
    out = layer.forward(xd, idd, wd)
    torch.cuda.synchronize()
    got, ref = values(out), bf16_linear.experts(x, ids, wt, w1, w2)
    assert np.all(np.isfinite(got)) and np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)
    if T > 5:
        assert not got[3].any()
    # the same bits from the grouped products called one by one
    _, offsets, order, pos = route(ids, E)
    h = torch.empty((T * k, I), dtype=BF, device="cuda")
    y = torch.zeros((T * k, H), dtype=BF, device="cuda")
    rows = torch.zeros(T * k, dtype=torch.int32, device="cuda")
    rows[:len(order)] = dev(order)
    _lib.moe_w4a4_grouped_linear_bf16(xd, layer.w1, dev(offsets), h, rows=rows, row_divisor=k, function=FN["silu"], gated=True)
    _lib.moe_w4a4_grouped_linear_bf16(h, layer.w2, dev(offsets), y)
    torch.cuda.synchronize()
    yv, want = values(y).astype(np.float32), np.zeros((T, H), np.float32)
    lo, hi = want.astype(np.float64), want.astype(np.float64)
    for r, p in enumerate(pos):
        if p >= 0:
            lo[r // k] += np.float64(wt[r // k, r % k]) * yv[p]
            hi[r // k] += np.abs(np.float64(wt[r // k, r % k]) * yv[p])
    tol = hi * k * 2.0 ** -23
    assert np.all(np.abs(got - lo) <= tol + (np.abs(lo) + tol) * 2.0 ** -8)
    # in the place of x, and on fewer tokens than the workspace holds
    wide = layer.with_capacity(T + 50)
    x2 = xd.clone()
    wide.forward(x2, idd, wd, out=x2)
    torch.cuda.synchronize()
    assert torch.equal(x2, out)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_experts_and_linears_captured_and_replayed(T):
    """Replayed three times on new inputs, with eager calls on the same workspace in between;
    every replay equals the eager call bit for bit."""
    log(f"[test] experts_bf16 T {T} in a graph")
    H, I, E, k = 256, 128, 16, 3
    rng = np.random.default_rng(8)
    layer, _, _ = make_experts(rng, H, I, E, k, T)
    mlp = Bf16MLP(Bf16Linear(dev_bf16(weights(rng, 2 * I, H)[0]), function=FN["silu"], gated=True),
                  Bf16Linear(dev_bf16(weights(rng, H, I)[0])))

    def inputs(seed):
        r = np.random.default_rng(seed)
        ids, wt = routing(r, T, E, k)
        return [dev_bf16(rows_like(r, T, H)[0]), dev(ids), dev(wt)]

    def call(a, out=None):
        out = layer.forward(*a, out=out)
        return mlp.forward(a[0], out=out, addend=out)

    sets = [inputs(1), inputs(2)]
    eager = [call(a) for a in sets]
    held, out = [t.clone() for t in sets[0]], torch.empty_like(eager[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(held, out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(held, out)
    for which in (1, 0, 1):
        for dst, src in zip(held, sets[which]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[which])
        assert torch.equal(call(sets[1 - which]), eager[1 - which])


def test_linears_at_the_same_time():
    """No workspace: one linear on two streams at once."""
    log("[test] one Bf16Linear on two streams")
    rng = np.random.default_rng(9)
    lin = Bf16Linear(dev_bf16(weights(rng, 512, 1024)[0]))
    xs = [dev_bf16(rows_like(rng, T, 1024)[0]) for T in (40, 600)]
    want = [lin.forward(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    for i in range(20):
        for x, s, o in zip(xs, streams, outs):
            lin.forward(x, out=o[i], stream=s.cuda_stream)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, t) for t in o)
