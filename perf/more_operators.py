"""Workloads of the bfloat16 operators around the routed-expert layer, for timing
and for comparing their kernels with plain torch.

Three operators, each with the calls a serving program makes of it.  They are
what a mixed-precision checkpoint keeps out of the 4-bit formats:

  linear   a dense product with bfloat16 weights, its bias, activation (gated or
           not), row scale and addend in the epilogue: router gates, shared
           experts, projections;
  grouped  the same product grouped by expert, rows sorted by expert in ragged
           groups and gathered on the way in: expert layers left unquantized;
  post     the norm after a block with its gate and residual scale, the addition
           to the residual stream, and the norm (and MXFP8 quantization) before the
           next block, in one pass.

Sizes are those of the repository's layer (hidden 4096, inter 2048, 256
experts, top-6; 1, 8, 512, 4096 and 16384 tokens) and ragged ones.

Eight-bit outputs come back as the values they stand for: E4M3 elements and
E8M0 scales as torch's types of that name.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- cases
def _linear(name, tokens, k, n, fn="none", gated=False, bias="none", rowscale=False, add="none", f32=False, pad=0):
    return dict(name=name, op="linear", tokens=tokens, k=k, n=n, fn=fn, gated=gated, bias=bias, rowscale=rowscale,
                add=add, f32=f32, pad=pad)


def _grouped(name, rows, experts, k, n, fn="none", gated=False, bias="none", gather=0, rowscale=False, f32=False,
             skew=0.0, spare=0):
    return dict(name=name, op="grouped", rows=rows, experts=experts, k=k, n=n, fn=fn, gated=gated, bias=bias,
                gather=gather, rowscale=rowscale, f32=f32, skew=skew, spare=spare)


def _post(name, rows, cols, norm=True, gate="none", f32=False, want_y=True, codes=False):
    return dict(name=name, op="post", rows=rows, cols=cols, norm=norm, gate=gate, f32=f32, want_y=want_y, codes=codes)


def listed():
    return [
        # one token's router logits in float32, from a gate kept in bfloat16
        _linear("linear_gate_1x4096x256", 1, 4096, 256, f32=True),
        # a decode batch through a shared expert's gate and up projections
        _linear("linear_decode_8x4096x2048", 8, 4096, 2048, fn="silu", gated=True),
        # sizes that fit no tile; a bias, a smooth activation, a float32 residual stream
        _linear("linear_ragged_333x1064x1111", 333, 1064, 1111, fn="gelu_tanh", bias="bf16", add="f32", pad=24),
        # a prefill's router logits: few outputs, a long sum
        _linear("linear_gate_4096x4096x256", 4096, 4096, 256, f32=True),
        # prefills through a shared expert: its down projection, weighted for each token and added to the routed
        # experts' output, and its gate and up projections
        _linear("linear_down_4096x2048x4096", 4096, 2048, 4096, rowscale=True, add="bf16"),
        _linear("linear_gate_up_16384x4096x2048", 16384, 4096, 2048, fn="silu", gated=True),
        # the gate and up projections of 8 tokens' six experts each: about 48 experts with one row
        _grouped("grouped_decode_48x4096x2048", 48, 256, 4096, 2048, fn="silu", gated=True, gather=6),
        # a few experts, some of them empty, sizes that fit no tile, rows behind the last expert's
        _grouped("grouped_ragged_1517x1000x777", 1517, 37, 1000, 777, fn="gelu", bias="f32", skew=1.2, f32=True, spare=13),
        # the down projection of a prefill's routed rows, weighted, popular and unpopular experts
        _grouped("grouped_down_98304x2048x4096", 98304, 256, 2048, 4096, rowscale=True, skew=0.7),
        # one token behind its block: both norms and a gate for each channel
        _post("post_decode_1x4096", 1, 4096, gate="channel"),
        # a batch with wide ragged rows, a gate for each row, a float32 residual stream, E4M3 codes
        _post("post_517x7200_f32", 517, 7200, gate="row", f32=True, codes=True),
        # a prefill whose consumer reads the quantized tokens alone
        _post("post_prefill_16384x4096", 16384, 4096, want_y=False, codes=True),
    ]


def _spread(rng, low, high):
    """A whole number from [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


FUNCTIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def draw(rng):
    op = rng.choice(("linear", "linear", "grouped", "grouped", "post"))
    if op == "post":
        cols = 32 * _spread(rng, 1, 512)
        rows = _spread(rng, 1, min(16384, (16384 * 4096) // cols))
        codes = rng.random() < 0.5
        return dict(op=op, rows=rows, cols=cols, norm=rng.random() < 0.8,
                    gate=rng.choice(("none", "channel", "row", "full")), f32=rng.random() < 0.4,
                    want_y=not codes or rng.random() < 0.5, codes=codes)
    gated = rng.random() < 0.4
    common = dict(fn=rng.choice(FUNCTIONS), gated=gated, bias=rng.choice(("none", "none", "bf16", "f32")),
                  rowscale=rng.random() < 0.3, f32=rng.random() < 0.3)
    if op == "linear":
        k, n = 8 * _spread(rng, 2, 1024), _spread(rng, 1, 8192)
        tokens = _spread(rng, 1, min(16384, (16384 * 4096 * 4096) // (k * n * (2 if gated else 1))))
        return dict(op=op, tokens=tokens, k=k, n=n, add=rng.choice(("none", "none", "bf16", "f32")),
                    pad=rng.choice((0, 0, 8, 72)), **common)
    experts, k, n = _spread(rng, 1, 256), 8 * _spread(rng, 2, 512), _spread(rng, 1, 4096)
    rows = _spread(rng, 1, min(98304, (16384 * 6 * 2048 * 2048) // (k * n)))
    return dict(op=op, rows=rows, experts=experts, k=k, n=n, gather=rng.choice((0, 1, 6)),
                skew=rng.choice((0.0, 0.7, 1.2)), spare=rng.choice((0, 0, 5)), **common)


def _counts(case):
    """Rows of the experts from the most to the least popular (which expert is which goes by the seed)."""
    weight = (1.0 + np.arange(case["experts"])) ** -case["skew"]
    g = np.random.default_rng([case["rows"], case["experts"], case["k"], int(10 * case["skew"])])
    return g.multinomial(case["rows"], weight / weight.sum())


def work(case):
    if case["op"] == "post":
        n = case["rows"] * case["cols"]
        gate = {"none": 0, "channel": 4 * case["cols"], "row": 4 * case["rows"], "full": 2 * n}[case["gate"]]
        return dict(bytes=n * (2 + 2 * (4 if case["f32"] else 2) + (2 if case["want_y"] else 0)
                               + (1 + 1 / 32 if case["codes"] else 0)) + gate + 4 * case["cols"] * (2 if case["norm"] else 1),
                    flops=12 * n)
    k, n, wide = case["k"], case["n"], 2 if case["gated"] else 1
    if case["op"] == "linear":
        t, groups, x_rows = case["tokens"], 1, case["tokens"]
        add = {"none": 0, "bf16": 2, "f32": 4}[case["add"]]
    else:
        t, groups, add = case["rows"], int((_counts(case) > 0).sum()), 0
        x_rows = -(-t // case["gather"]) if case["gather"] else t
    bias = {"none": 0, "bf16": 2, "f32": 4}[case["bias"]]
    return dict(bytes=2 * x_rows * k + groups * wide * n * (2 * k + bias) + t * n * ((4 if case["f32"] else 2) + add)
                + (4 * t if case["rowscale"] else 0), flops=2 * t * k * n * wide)


# ---------------------------------------------------------------- inputs
def _rows(g, rows, cols):
    """Activations as a residual stream has them: a scale for each channel,
    a few channels far above the others, rows of unequal size."""
    chan = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    chan[torch.randint(0, cols, (max(1, cols // 512),), generator=g, device="cuda")] *= 20.0
    row = torch.exp(0.3 * torch.randn(rows, 1, generator=g, device="cuda"))
    return (torch.randn(rows, cols, generator=g, device="cuda") * chan * row).to(torch.bfloat16)


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")   # noqa: E731
    s = dict(case=case)
    if case["op"] == "post":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _rows(g, rows, cols)
        s["residual"] = 4 * _rows(g, rows, cols)
        if case["f32"]:
            s["residual"] = s["residual"].float() + 0.01 * normal(rows, cols)
        s["post_weight"] = 1 + 0.1 * normal(cols) if case["norm"] else None
        s["next_weight"] = 1 + 0.1 * normal(cols)
        s["gate"] = {"none": lambda: None, "channel": lambda: 0.5 + 0.1 * normal(cols),
                     "row": lambda: torch.sigmoid(normal(rows, 1)),
                     "full": lambda: torch.sigmoid(normal(rows, cols)).to(torch.bfloat16)}[case["gate"]]()
        s["residual_out"] = torch.empty_like(s["residual"])
        s["y"] = torch.empty_like(s["x"]) if case["want_y"] else None
        s["codes"] = torch.empty((rows, cols), dtype=torch.uint8, device="cuda") if case["codes"] else None
        s["scales"] = torch.empty((rows, cols // 32), dtype=torch.uint8, device="cuda") if case["codes"] else None
        return s
    k, n, wide = case["k"], case["n"], 2 if case["gated"] else 1
    size = 1.0 / math.sqrt(k)
    if case["op"] == "linear":
        t = case["tokens"]
        s["x"] = _rows(g, t, k + case["pad"])[:, :k]      # (a slice of wider rows)
        s["w"] = (size * normal(wide * n, k)).to(torch.bfloat16)
        s["bias"] = None if case["bias"] == "none" else (0.1 * normal(wide * n)).to(TYPES[case["bias"]])
        s["addend"] = None if case["add"] == "none" else normal(t, n).to(TYPES[case["add"]])
    else:
        t, e = case["rows"], case["experts"]
        order = torch.randperm(e, generator=g, device="cuda").cpu().numpy()
        counts = np.zeros(e, np.int64)
        counts[order] = _counts(case)
        s["bounds"] = [0] + np.cumsum(counts).tolist()     # the plain form's loop runs over these
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda")
        s["rows"] = None
        if case["gather"]:                                 # routed rows r = token * top-k + slot, rising within an expert
            slots = torch.randperm(t, generator=g, device="cuda")
            group = torch.repeat_interleave(torch.arange(e, device="cuda"), torch.tensor(counts, device="cuda"))
            s["rows"] = torch.sort(group * t + slots).values.remainder(t).to(torch.int32)
            if case["spare"]:
                s["rows"] = torch.cat([s["rows"], torch.full((case["spare"],), -1, dtype=torch.int32, device="cuda")])
        s["x"] = _rows(g, -(-t // case["gather"]) if case["gather"] else t + case["spare"], k)
        s["w"] = torch.empty((e, wide * n, k), dtype=torch.bfloat16, device="cuda")
        for i in range(e):
            s["w"][i] = size * normal(wide * n, k)
        s["bias"] = None if case["bias"] == "none" else (0.1 * normal(e, wide * n)).to(TYPES[case["bias"]])
        t += case["spare"]                                 # rows behind the last expert's, which stay as they are
    s["rowscale"] = torch.sigmoid(normal(t)) if case["rowscale"] else None
    s["out"] = torch.zeros((t, n), dtype=torch.float32 if case["f32"] else torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- the framework's operators
def _run_own(s):
    import block_scaled_fp4_pre_amd as amd
    case = s["case"]
    if case["op"] == "post":
        amd.moe_w4a4_post_norm(s["x"], s["residual"], s["residual_out"], EPS, post_weight=s["post_weight"],
                               gate=s["gate"], scale=0.7, next_weight=s["next_weight"], y=s["y"], codes=s["codes"],
                               scales=s["scales"], mma_type=amd.MOE_MMA_FP8_X_MXF4)
        return _post_outputs(s)
    fn = dict(none=amd.MOE_FN_NONE, relu=amd.MOE_FN_RELU, silu=amd.MOE_FN_SILU, gelu=amd.MOE_FN_GELU,
              gelu_tanh=amd.MOE_FN_GELU_TANH)[case["fn"]]
    if case["op"] == "linear":
        amd.moe_w4a4_linear_bf16(s["x"], s["w"], s["out"], bias=s["bias"], function=fn, gated=case["gated"],
                                 row_scale=s["rowscale"], addend=s["addend"])
    else:
        amd.moe_w4a4_grouped_linear_bf16(s["x"], s["w"], s["offsets"], s["out"], rows=s["rows"],
                                         row_divisor=max(1, case["gather"]), bias=s["bias"], function=fn,
                                         gated=case["gated"], row_scale=s["rowscale"])
    return dict(out=s["out"])


def _post_outputs(s):
    return dict(residual=s["residual_out"], y=s["y"],
                elements=None if s["codes"] is None else s["codes"].view(torch.float8_e4m3fn),
                scales=None if s["codes"] is None else s["scales"].view(torch.float8_e8m0fnu))


# ---------------------------------------------------------------- the plain forms
def _power(e):
    """2^e in float32 from its bits, e in [-127, 127] (a library's power may be a last bit off)."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantize(v):
    """E4M3 elements and power-of-two scales, one per 32, the smallest with amax <= 448 * scale."""
    groups = v.float().unflatten(-1, (-1, 32))
    part, power = torch.frexp(groups.abs().amax(-1))          # amax = part * 2^power, part in [0.5, 1)
    e = torch.where(part == 0, -127, (power - 9 + (part > 0.875)).clamp(-127, 127))
    scaled = groups * _power(-e).unsqueeze(-1)
    step = (torch.frexp(scaled).exponent - 1).clamp(min=-6) - 3
    return (torch.round(scaled * _power(-step)) * _power(step)).flatten(-2), _power(e)


def _function(v, fn):
    if fn == "relu":
        return torch.where(v > 0, v, 0.0)
    if fn == "silu":
        return v / (1 + torch.exp(-v))
    if fn == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if fn == "gelu_tanh":                                     # 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _product(case, x, w, bias):
    v = x.float() @ w.float().T
    if bias is not None:
        v = v + bias.float()
    if case["gated"]:
        return _function(v[:, :case["n"]], case["fn"]) * v[:, case["n"]:]
    return _function(v, case["fn"])


def _run_plain(s):
    case = s["case"]
    if case["op"] == "post":
        # sums and norms in 64 bits: the quantizer behind them turns a last bit next to a border into a whole step
        z = s["x"].double()
        if s["post_weight"] is not None:
            z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + EPS) * s["post_weight"].double()
        if s["gate"] is not None:
            z = z * s["gate"].double()
        # (the factor is a float32)
        h = (s["residual"].double() + float(np.float32(0.7)) * z).float().to(s["residual"].dtype)
        d = h.double()
        y = (d / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS) * s["next_weight"].double()).float().to(torch.bfloat16)
        elements, scale = _quantize(y) if case["codes"] else (None, None)
        return dict(residual=h, y=y if case["want_y"] else None,
                    elements=None if elements is None else elements.to(torch.float8_e4m3fn),
                    scales=None if scale is None else scale.to(torch.float8_e8m0fnu))
    if case["op"] == "linear":
        v = _product(case, s["x"], s["w"], s["bias"])
        if s["rowscale"] is not None:
            v = v * s["rowscale"].unsqueeze(-1)
        if s["addend"] is not None:
            v = v + s["addend"].float()
        return dict(out=v.to(s["out"].dtype))
    for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if a == b:
            continue
        x = s["x"][a:b] if s["rows"] is None else s["x"][(s["rows"][a:b] // case["gather"]).long()]
        v = _product(case, x, s["w"][e], None if s["bias"] is None else s["bias"][e])
        if s["rowscale"] is not None:
            v = v * s["rowscale"][a:b].unsqueeze(-1)
        s["out"][a:b] = v.to(s["out"].dtype)
    return dict(out=s["out"])


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---------------------------------------------------------------- 64-bit values
def _two_to(e):
    """2^e in float64, e whole."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest(v):
    """E4M3 elements (by a search among the format's magnitudes) and scales of float64 values."""
    codes = torch.arange(127, device="cuda")
    m, p = (codes % 8).double(), codes // 8
    grid = torch.where(p == 0, m * 2.0 ** -9, (1 + m / 8) * _two_to(p - 7))
    groups = v.reshape(v.shape[0], -1, 32)
    amax = groups.abs().max(-1).values
    e = torch.full_like(amax, -127.0)
    guess = torch.floor(torch.log2(amax / grid[-1]))
    for k in (1, 0, -1):                                       # the smallest of the powers around the quotient that holds amax
        fits = (amax > 0) & (_two_to((guess + k).clamp(min=-1000)) * grid[-1] >= amax)
        e = torch.where(fits, guess + k, e)
    scale = _two_to(e.clamp(-127, 127))
    mag = (groups / scale.unsqueeze(-1)).abs()
    up = torch.searchsorted(grid, mag.contiguous()).clamp(1, len(grid) - 1)
    to_low, to_up = mag - grid[up - 1], grid[up] - mag
    pick = torch.where((to_up < to_low) | ((to_up == to_low) & (up % 2 == 0)), up, up - 1)
    return torch.where(groups < 0, -grid[pick], grid[pick]).reshape(v.shape), scale


def _exact_function(v, fn):
    return {"none": lambda: v, "relu": lambda: torch.clamp(v, min=0), "silu": lambda: v * torch.special.expit(v),
            "gelu": lambda: v * torch.special.ndtr(v),
            "gelu_tanh": lambda: 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * v * (1 + 0.044715 * v ** 2)))}[fn]()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "post":
        z, cols = s["x"].double(), case["cols"]
        if case["norm"]:
            z = z * s["post_weight"].double() * torch.rsqrt(torch.linalg.vector_norm(z, dim=-1, keepdim=True) ** 2 / cols + EPS)
        step = z if s["gate"] is None else torch.mul(z, s["gate"].double())
        total = torch.add(s["residual"].double(), step, alpha=float(np.float32(0.7)))
        h = total.to(torch.float32).to(s["residual"].dtype).double()
        y = h * s["next_weight"].double() / torch.sqrt(torch.linalg.vector_norm(h, dim=-1, keepdim=True) ** 2 / cols + EPS)
        elements, scales = _nearest(y.to(torch.float32).to(torch.bfloat16).double()) if case["codes"] else (None, None)
        return dict(residual=total, y=y if case["want_y"] else None, elements=elements, scales=scales)
    n = case["n"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    groups = [(0, case["tokens"])] if case["op"] == "linear" else list(zip(s["bounds"], s["bounds"][1:]))
    for e, (a, b) in enumerate(groups):
        if b <= a:
            continue
        at = torch.arange(a, b, device="cuda")
        if case["op"] == "grouped" and case["gather"]:
            at = torch.div(s["rows"][a:b].long(), case["gather"], rounding_mode="floor")
        w = s["w"] if case["op"] == "linear" else s["w"][e]
        v = torch.matmul(s["x"].index_select(0, at).double(), w.double().t())
        if s["bias"] is not None:
            v += (s["bias"] if case["op"] == "linear" else s["bias"][e]).double()
        v = torch.mul(_exact_function(v[:, :n], case["fn"]), v[:, n:]) if case["gated"] else _exact_function(v, case["fn"])
        if case["rowscale"]:
            v = torch.mul(v, s["rowscale"][a:b, None].double())
        out[a:b] = v if case["op"] == "grouped" or s["addend"] is None else v + s["addend"].double()
    return dict(out=out)
