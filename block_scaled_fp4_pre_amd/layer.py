"""MoeW4A4Layer: owns the device buffers of one layer and calls the C ABI.

PyTorch provides the device memory and the stream; every computation runs in
the library's HIP kernels.  Weights can be loaded either as canonical MXFP4
(codes + scale bytes) or as fp32 matrices, which are quantized on the device by
moe_w4a4_quantize and then re-laid by moe_w4a4_prepare_weights.  An NVFP4
layer (MOE_MMA_NVF4_X_NVF4) takes NVFP4 codes, E4M3 scale bytes per 16 and the
tensor scales instead (moe_w4a4_quantize_nvfp4, moe_w4a4_prepare_weights_nvfp4).
MoeW4A4Layer.forward_block runs the layer behind its norm and router; W4A4Linear
is a dense linear on the same formats.  Bf16Linear, Bf16MLP and Bf16Experts are what a
checkpoint keeps in bfloat16: gates and projections, shared experts, whole expert
layers (with the same forward and forward_block).
"""
from __future__ import annotations

import concurrent.futures
import contextlib
import ctypes

import torch

from . import _lib


def _torch_stream(stream, device):
    """torch's stream of a raw handle.  0 is the default stream's (torch would take
    an external stream of handle 0 to mean a new stream of its pool)."""
    handle = int(stream)
    return torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)


def _output(shape, dtype, device, stream):
    """A new tensor for a call to fill on `stream` (None: the current stream).
    It is of that stream's memory: the current stream's own free blocks may have
    pending work of that stream on them.  The caller reads it on the current
    stream, so its memory waits for that one too before it is used again."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(torch.cuda.current_stream(device))
    return out


class _Block:
    """forward_block of the expert layers (H, E, k, max_tokens, mma_type, device)."""

    def _codes(self, T):
        """Where the norm is to leave its codes and scales (None: the experts quantize)."""
        return None, None

    def _experts(self, T, y, codes, ids, weights, out) -> None:
        """The routed experts of y (or of the codes _codes gave) into out, on the current stream."""
        raise NotImplementedError

    def _held(self):
        """The layer's own tensors that `_experts` refuses as its output."""
        return ()

    def _check_block(self, T, gate, bias, scoring, num_groups, topk_groups, scale, shared, residual_out, out,
                     post=(None, None, None, None), x=None) -> None:
        """Everything that the steps behind the norm would refuse: the norm may
        overwrite x and the residual, so the others' arguments are checked first."""
        H, E, dev = self.H, self.E, self.device.index
        if T > self.max_tokens:
            raise ValueError(f"x: {T} tokens, the layer holds {self.max_tokens}")
        for name, lin, n in (("gate_weight", gate, E), ("shared", shared, H)):
            if not isinstance(lin, (W4A4Linear, Bf16Linear, Bf16MLP)):
                continue
            if (lin.K, lin.N, lin.device) != (H, n, self.device):
                raise ValueError(f"{name}: from {lin.K} to {lin.N} on {lin.device}, expected {H} to {n} on {self.device}")
            if isinstance(lin, W4A4Linear) and lin.max_tokens < T:
                raise ValueError(f"{name}: holds {lin.max_tokens} tokens, not {T}")
            if not isinstance(lin, W4A4Linear):
                widest = max(lin.gate_up.N, lin.N) if isinstance(lin, Bf16MLP) else lin.N
                most = min(_lib.MOE_BF16_MAX_ROWS, _lib.MOE_BF16_MAX_OUT // widest)
                if T > most:
                    raise ValueError(f"{name}: takes {most} tokens, not {T}")
        if not isinstance(gate, (W4A4Linear, Bf16Linear)):
            _lib._fits(gate, "gate_weight", (torch.bfloat16,), (E, H), dev, contiguous=False)
        if shared is not None and not isinstance(shared, (W4A4Linear, Bf16Linear, Bf16MLP)):
            raise ValueError(f"shared: expected a W4A4Linear, Bf16Linear or Bf16MLP, got {type(shared).__name__}")
        _lib._check_router_config(E, self.k, scoring, num_groups, topk_groups, scale)
        if bias is not None:
            _lib._fits(bias, "bias", (torch.float32,), (E,), dev)
        post_weight, post_gate, post_scale, next_weight = post
        after = any(v is not None for v in post)
        if after:
            types = (torch.bfloat16, torch.float32)
            for name, w in (("post_weight", post_weight), ("next_weight", next_weight)):
                if w is not None and _lib._fits(w, name, types, (H,), dev) % 16:
                    raise ValueError(f"{name}: not 16-byte aligned")
            if post_weight is not None and next_weight is not None and post_weight.dtype is not next_weight.dtype:
                raise ValueError(f"next_weight: {next_weight.dtype}, post_weight: {post_weight.dtype}")
            if post_gate is not None:
                kind = _lib._gate_kind(post_gate, T, H)
                place = _lib._fits(post_gate, "post_gate", types, ((H,), (T, 1), (T, H))[kind - 1], dev)
                if place % 16 and kind != _lib.MOE_GATE_ROW:
                    raise ValueError("post_gate: not 16-byte aligned")
            places = [t.data_ptr() for t in (residual_out, out) if t is not None and T > 0]
            for name, t in (("post_weight", post_weight), ("post_gate", post_gate), ("next_weight", next_weight)):
                if t is not None and t.data_ptr() in places:
                    raise ValueError(f"{name}: in the place of an output")
            if post_scale is not None and not abs(post_scale) <= 3.402823466e38:
                raise ValueError(f"post_scale: {post_scale}")
        if out is not None:
            # (a forward alone takes more rows, and bit patterns)
            plain = shared is None and not after and isinstance(self, MoeW4A4Layer)
            rows = max(T, out.shape[0] if out.dim() == 2 else 0) if plain else T
            types = (torch.bfloat16, torch.int16, torch.uint16) if plain else (torch.bfloat16,)
            place = _lib._fits(out, "out", types, (rows, H), dev)
            if place % 16:
                raise ValueError("out: not 16-byte aligned")
            if residual_out is not None and place == residual_out.data_ptr() and T > 0:
                raise ValueError("out: in the place of residual_out")
            if after and x is not None and place == x.data_ptr() and T > 0:
                raise ValueError("out: in the place of x, the residual stream")
            for t in (*self._held(), *(shared._held() if shared is not None else ())):
                if t is not None and place == t.data_ptr() and T > 0:
                    raise ValueError("out: in the place of weights or a workspace")

    def forward_block(self, x, residual, norm_weight, eps, gate_weight, residual_out=None, bias=None,
                      scoring=_lib.MOE_SCORE_SOFTMAX, num_groups=1, topk_groups=1, renormalize=True, scale=1.0,
                      shared=None, out=None, stream=None, post_weight=None, post_gate=None, post_scale=None,
                      next_weight=None):
        """One decoder block's feed-forward half: residual addition and norm
        (moe_w4a4_add_rmsnorm), router logits, the router's choice
        (moe_w4a4_router), the routed experts, and a shared linear or MLP if there
        is one.  Returns (out, h): out = experts(y) (+ shared(y)) bf16 [T, H], and
        the new residual stream h = x + residual, of the residual's type.
        With any of post_weight, post_gate, post_scale and next_weight the block ends
        with moe_w4a4_post_norm, and returns (y', h'): h' = h + post_scale * post_gate *
        (the norm of out under post_weight), and y' = the norm of h' under next_weight,
        what the next block reads (None without one), both norms with eps.
        x bf16 [T, H]; residual bf16 / float32 [T, H] (residual_out like it,
        may be it; a new tensor if None), or None (h is x then, and residual_out
        None); norm_weight [H].
        gate_weight: bf16 [E, H], whose logits are torch's own product and so
        rounded to bf16 before the choice; or a W4A4Linear or Bf16Linear with
        out_features E, whose logits are float32.  bias float32 [E].
        shared: a W4A4Linear, Bf16Linear or Bf16MLP from H to H, whose sum is added
        to the experts' output, that one rounded to bf16, and rounded again.
        Past the fused pre-dispatch (more than 8192 routed rows) the norm
        quantizes y into the workspace and the experts start from that; a
        W4A4Linear gate or `shared` quantizes y for itself.
        Arguments that any step would refuse raise before the first launch, with
        x and residual as they were."""
        T = x.shape[0]
        post = (post_weight, post_gate, post_scale, next_weight)
        self._check_block(T, gate_weight, bias, scoring, num_groups, topk_groups, scale, shared, residual_out, out, post,
                          x if residual is None else None)
        caller = None if stream is None else torch.cuda.current_stream(self.device)
        on_stream = contextlib.nullcontext() if stream is None else torch.cuda.stream(_torch_stream(stream, self.device))
        if residual_out is None and residual is not None:
            residual_out = _output(residual.shape, residual.dtype, self.device, stream)
        if out is None:
            out = _output((T, self.H), torch.bfloat16, self.device, stream)
        with torch.cuda.device(self.device), on_stream:
            y = torch.empty((T, self.H), dtype=torch.bfloat16, device=self.device)
            ids = torch.empty((T, self.k), dtype=torch.int32, device=self.device)
            weights = torch.empty((T, self.k), dtype=torch.float32, device=self.device)
            codes, scales = self._codes(T)
            _lib.moe_w4a4_add_rmsnorm(x, residual, norm_weight, eps, residual_out=residual_out, y=y, codes=codes,
                                      scales=scales, mma_type=self.mma_type)
            if isinstance(gate_weight, (W4A4Linear, Bf16Linear)):
                logits = gate_weight.forward(y, dtype=torch.float32)
            else:
                # (autocast may ask for another type, which the router would refuse)
                with torch.autocast("cuda", enabled=False) if torch.is_autocast_enabled() else contextlib.nullcontext():
                    logits = torch.nn.functional.linear(y, gate_weight)
            _lib.moe_w4a4_router(logits, ids, weights, bias=bias, scoring=scoring, num_groups=num_groups,
                                 topk_groups=topk_groups, renormalize=renormalize, scale=scale)
            self._experts(T, y, codes, ids, weights, out)
            if shared is not None:
                shared.forward(y, out=out, addend=out)
            if all(v is None for v in post):
                return out, x if residual is None else residual_out
            h = x if residual is None else residual_out
            if residual_out is None:
                residual_out = torch.empty_like(x)
                if caller is not None:
                    residual_out.record_stream(caller)
            _lib.moe_w4a4_post_norm(out, h, residual_out, eps, post_weight=post_weight, gate=post_gate,
                                    scale=1.0 if post_scale is None else post_scale, next_weight=next_weight,
                                    y=None if next_weight is None else out)
        return None if next_weight is None else out, residual_out


class MoeW4A4Layer(_Block):
    PREDISPATCH_ROWS = 8192      # routed rows up to which a forward quantizes and routes in one launch

    def __init__(self, hidden: int, inter: int, num_experts: int, topk: int, max_tokens: int,
                 device: str | torch.device = "cuda", mma_type: int = _lib.MOE_MMA_MXF4_X_MXF4,
                 prepared: torch.Tensor | None = None):
        """mma_type: MOE_MMA_MXF4_X_MXF4 (MXFP4 activations) or MOE_MMA_FP8_X_MXF4
        (MXFP8 E4M3 activations), the weights MXFP4 in both; or
        MOE_MMA_NVF4_X_NVF4 (NVFP4 activations and weights).  prepared: an
        existing prepared-weights buffer of the same shape to share (see
        with_capacity), else a new one is allocated."""
        self.H, self.I, self.E, self.k, self.max_tokens = hidden, inter, num_experts, topk, max_tokens
        self.mma_type = mma_type
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.cfg = _lib.make_cfg(hidden, inter, num_experts, topk, max_tokens, mma_type=mma_type)
        pb, wb = _lib.moe_w4a4_query(self.cfg)
        if prepared is None:
            prepared = torch.empty(pb, dtype=torch.uint8, device=self.device)
        elif prepared.numel() * prepared.element_size() < pb or prepared.device != self.device:
            raise ValueError("shared prepared buffer is too small or on another device")
        self.prepared = prepared
        self.workspace = torch.empty(wb, dtype=torch.uint8, device=self.device)
        self.layout = _lib.moe_w4a4_workspace_layout(self.cfg)
        # the single-launch forward's state region: zero before its first call
        # (every call leaves it zero)
        m = self.layout["mega"]
        self.workspace[m:m + _lib.MOE_MEGA_STATE_BYTES].zero_()

    @property
    def nvfp4(self) -> bool:
        return self.mma_type == _lib.MOE_MMA_NVF4_X_NVF4

    def with_capacity(self, max_tokens: int, mma_type: int | None = None) -> "MoeW4A4Layer":
        """A layer over the same prepared weights (shared, not copied) with its
        own workspace for max_tokens tokens; mma_type may switch between the
        two MX types, which use the same MXFP4 weights."""
        mma = self.mma_type if mma_type is None else mma_type
        if (mma == _lib.MOE_MMA_NVF4_X_NVF4) != self.nvfp4:
            raise ValueError("NVFP4 and MXFP4 layers cannot share prepared weights")
        return MoeW4A4Layer(self.H, self.I, self.E, self.k, max_tokens, self.device, mma, prepared=self.prepared)

    # ---- weights ------------------------------------------------------------
    def canonical_buffers(self):
        H, I, E, G = self.H, self.I, self.E, _lib.scale_group(self.cfg)
        u8 = dict(dtype=torch.uint8, device=self.device)
        return (torch.empty((E, 2 * I, H // 2), **u8), torch.empty((E, 2 * I, H // G), **u8),
                torch.empty((E, H, I // 2), **u8), torch.empty((E, H, I // G), **u8))

    def load_canonical(self, w1_codes, w1_scales, w2_codes, w2_scales, tensor_scales=None) -> None:
        """tensor_scales (NVFP4 only): (g_x, g_h, g_w1 fp32 [E], g_w2 fp32 [E])."""
        if self.nvfp4:
            gx, gh, gw1, gw2 = tensor_scales
            gw1 = torch.as_tensor(gw1, dtype=torch.float32).to(self.device)
            gw2 = torch.as_tensor(gw2, dtype=torch.float32).to(self.device)
            _lib.moe_w4a4_prepare_weights_nvfp4(self.cfg, w1_codes, w1_scales, gw1, w2_codes, w2_scales, gw2,
                                                gx, gh, self.prepared)
            torch.cuda.current_stream(self.device).synchronize()   # gw1/gw2 are temporaries
        else:
            assert tensor_scales is None
            _lib.moe_w4a4_prepare_weights(self.cfg, w1_codes, w1_scales, w2_codes, w2_scales, self.prepared)

    def quantize_fp32_weights(self, expert_source, threads: int = 16, weight_scales=None):
        """expert_source(e) -> (W1 [2I, H], W2 [H, I]) fp32 arrays (host or device).
        Returns the canonical buffers (w1c, w1s, w2c, w2s) on the device: MXFP4,
        or NVFP4 with weight_scales = (g_w1 [E], g_w2 [E]) the tensor scales."""
        bufs = self.canonical_buffers()
        w1c, w1s, w2c, w2s = bufs
        with concurrent.futures.ThreadPoolExecutor(max(1, threads)) as ex:
            futs = [ex.submit(expert_source, e) for e in range(min(self.E, 2 * threads))]
            nxt = len(futs)
            for e in range(self.E):
                w1, w2 = futs[e].result()
                futs[e] = None
                if nxt < self.E:
                    futs.append(ex.submit(expert_source, nxt))
                    nxt += 1
                d1 = torch.as_tensor(w1).to(self.device, torch.float32)
                d2 = torch.as_tensor(w2).to(self.device, torch.float32)
                if self.nvfp4:
                    _lib.moe_w4a4_quantize_nvfp4(d1, float(weight_scales[0][e]), w1c[e], w1s[e])
                    _lib.moe_w4a4_quantize_nvfp4(d2, float(weight_scales[1][e]), w2c[e], w2s[e])
                else:
                    _lib.moe_w4a4_quantize(d1, w1c[e], w1s[e])
                    _lib.moe_w4a4_quantize(d2, w2c[e], w2s[e])
        return bufs

    def load_fp32(self, expert_source, threads: int = 16, keep_canonical: bool = False, tensor_scales=None):
        """tensor_scales (NVFP4 only): (g_x, g_h, g_w1 [E], g_w2 [E])."""
        bufs = self.quantize_fp32_weights(expert_source, threads,
                                          None if tensor_scales is None else tensor_scales[2:])
        self.load_canonical(*bufs, tensor_scales=tensor_scales)
        if keep_canonical:
            return bufs
        del bufs
        return None

    # ---- forward ------------------------------------------------------------
    def forward(self, x, topk_ids, topk_weights, out=None, stream=None):
        """x bf16 [T, H]; topk_ids int32 [T, k] (ids outside [0, E) are skipped);
        topk_weights float32 [T, k]; out bf16 [T, H] or None.  Every tensor must
        be on the layer's device; anything else raises ValueError before a
        kernel is launched."""
        T = x.shape[0]
        if out is None:
            out = _output((T, self.H), torch.bfloat16, self.device, stream)
        with torch.cuda.device(self.device):
            _lib.moe_w4a4_forward(self.cfg, self.prepared, T, x, topk_ids, topk_weights, out, self.workspace,
                                  stream=stream)
        return out

    def forward_mega(self, x, topk_ids, topk_weights, out=None, stream=None):
        """The forward as one kernel launch (moe_w4a4_forward_mega: MXFP4 or
        fp8xfp4, at most 256 routed rows); arguments as forward."""
        T = x.shape[0]
        if out is None:
            out = _output((T, self.H), torch.bfloat16, self.device, stream)
        with torch.cuda.device(self.device):
            _lib.moe_w4a4_forward_mega(self.cfg, self.prepared, T, x, topk_ids, topk_weights, out, self.workspace,
                                       stream=stream)
        return out

    # ---- the steps of forward_block ------------------------------------------
    def _codes(self, T):
        if T * self.k <= self.PREDISPATCH_ROWS or self.nvfp4:
            return None, None
        wide = self.H if self.mma_type == _lib.MOE_MMA_FP8_X_MXF4 else self.H // 2
        return (self.ws("xq", (self.max_tokens, wide), torch.uint8)[:T],
                self.ws("xsf", (self.max_tokens, self.H // 32), torch.uint8)[:T])

    def _experts(self, T, y, codes, ids, weights, out) -> None:
        if codes is None:
            _lib.moe_w4a4_forward(self.cfg, self.prepared, T, y, ids, weights, out, self.workspace)
        else:
            _lib.moe_w4a4_run_stages(self.cfg, self.prepared, T, None, ids, weights, out, self.workspace,
                                     _lib.MOE_STAGE_ALL & ~_lib.MOE_STAGE_QUANT)

    def run_stages(self, stages, num_tokens, x=None, topk_ids=None, topk_weights=None, out=None,
                   gemm1_acc=None, stream=None):
        with torch.cuda.device(self.device):
            _lib.moe_w4a4_run_stages(self.cfg, self.prepared, num_tokens, x, topk_ids, topk_weights, out,
                                     self.workspace, stages, gemm1_acc=gemm1_acc, stream=stream)

    def ws(self, name: str, shape, dtype) -> torch.Tensor:
        """A view of one intermediate region of the workspace (see moe_w4a4_ws_layout)."""
        off = self.layout[name]
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.workspace[off:off + nbytes].view(dtype).view(*shape)


class W4A4Linear:
    """A dense linear with MXFP4 weights (moe_w4a4_linear): owns the prepared
    weights and the workspace for max_tokens tokens.  Calls that may run at the
    same time (on two streams, or in two captured graphs) need a linear each
    (with_capacity): they would share the workspace."""

    def __init__(self, in_features: int, out_features: int, max_tokens: int,
                 device: str | torch.device = "cuda", mma_type: int = _lib.MOE_MMA_MXF4_X_MXF4,
                 prepared: torch.Tensor | None = None):
        """mma_type: MOE_MMA_MXF4_X_MXF4 (tokens quantized to MXFP4) or
        MOE_MMA_FP8_X_MXF4 (MXFP8 E4M3).  prepared: the weights of another
        linear of the same shape to share (see with_capacity)."""
        self.K, self.N, self.max_tokens, self.mma_type = in_features, out_features, max_tokens, mma_type
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"expected a GPU, got {self.device}")
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.cfg = _lib.make_linear_cfg(in_features, out_features, max_tokens, mma_type)
        pb, wb = _lib.moe_w4a4_linear_query(self.cfg)
        if prepared is None:
            prepared = torch.empty(pb, dtype=torch.uint8, device=self.device)
        elif (not prepared.is_contiguous() or prepared.numel() * prepared.element_size() < pb
              or prepared.device != self.device):
            raise ValueError("shared prepared buffer is too small, not contiguous or on another device")
        self.prepared = prepared
        self.workspace = torch.empty(max(wb, 1), dtype=torch.uint8, device=self.device)
        self._cfg_ref, self._workspace_bytes = ctypes.byref(self.cfg), wb

    def with_capacity(self, max_tokens: int, mma_type: int | None = None) -> "W4A4Linear":
        """A linear over the same prepared weights with its own workspace."""
        return W4A4Linear(self.K, self.N, max_tokens, self.device,
                          self.mma_type if mma_type is None else mma_type, prepared=self.prepared)

    def _held(self):
        """Its own tensors that may not be its output."""
        return self.prepared, self.workspace

    def load_canonical(self, codes, scales) -> None:
        """codes uint8 [N, K/2] and scales uint8 [N, K/32], MXFP4 (moe_w4a4_quantize)."""
        with torch.cuda.device(self.device):
            _lib.moe_w4a4_linear_prepare(self.cfg, codes, scales, self.prepared)

    def load_fp32(self, weight) -> None:
        """weight [N, K] (host or device), quantized to MXFP4 on the device."""
        w = torch.as_tensor(weight).to(self.device, torch.float32).contiguous()
        codes = torch.empty((self.N, self.K // 2), dtype=torch.uint8, device=self.device)
        scales = torch.empty((self.N, self.K // 32), dtype=torch.uint8, device=self.device)
        with torch.cuda.device(self.device):
            _lib.moe_w4a4_quantize(w, codes, scales)
            _lib.moe_w4a4_linear_prepare(self.cfg, codes, scales, self.prepared)

    def _run(self, x, xq, xsf, out, addend, dtype, stream):
        if out is None:
            T = (x if x is not None else xq).shape[0]
            out = _output((T, self.N), dtype, self.device, stream)
        index = self.device.index
        if torch._C._cuda_getDevice() != index:
            with torch.cuda.device(index):
                return self._run(x, xq, xsf, out, addend, dtype, stream)
        _lib._linear_call(self._cfg_ref, self.K, self.N, self.mma_type, index, self.prepared.data_ptr(), x, out,
                          self.workspace.data_ptr(), self._workspace_bytes, xq, xsf, addend, stream)
        return out

    def forward(self, x, out=None, addend=None, dtype=torch.bfloat16, stream=None):
        """x bf16 [T, K] -> out [T, N] (bf16 or float32; made of `dtype` if
        None); addend bf16 [T, N] is added before the rounding (may be out)."""
        return self._run(x, None, None, out, addend, dtype, stream)

    def forward_quantized(self, codes, scales, out=None, addend=None, dtype=torch.bfloat16, stream=None):
        """The same from tokens quantized before (moe_w4a4_add_rmsnorm, moe_w4a4_quantize)."""
        return self._run(None, codes, scales, out, addend, dtype, stream)


def _gpu(device) -> torch.device:
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"expected a GPU, got {device}")
    return device if device.index is not None else torch.device("cuda", torch.cuda.current_device())


class Bf16Linear:
    """A dense linear with bfloat16 weights (moe_w4a4_linear_bf16): holds the weight, [N, K]
    or gated [2N, K] (gate rows, then up rows), and its bias.  No workspace: calls may
    run at the same time."""

    def __init__(self, weight, bias=None, function: int = _lib.MOE_FN_NONE, gated: bool = False):
        if not weight.is_cuda or weight.dtype is not torch.bfloat16 or weight.dim() != 2 or not weight.is_contiguous():
            raise ValueError("weight: expected a contiguous bfloat16 matrix on a GPU")
        if weight.data_ptr() % 16:
            raise ValueError("weight: not 16-byte aligned")
        wide, self.K = weight.shape
        if gated and wide % 2:
            raise ValueError(f"weight: {wide} rows, a gated linear has as many gate as up rows")
        self.N = wide // 2 if gated else wide
        self.device = weight.device
        _lib._check_linear_bf16_config(self.K, self.N, function)
        if bias is not None:
            _lib._fits(bias, "bias", (torch.bfloat16, torch.float32), (wide,), self.device.index)
        self.weight, self.bias, self.function, self.gated = weight, bias, function, gated

    def _held(self):
        """Its own tensors that may not be its output."""
        return self.weight, self.bias

    def forward(self, x, out=None, addend=None, row_scale=None, dtype=torch.bfloat16, stream=None):
        """x bf16 [T, K] -> out [T, N] (bf16 or float32; made of `dtype` if None):
        (addend +) (row_scale *) f(x W^T + bias); addend [T, N] may be out."""
        if out is None:
            out = _output((x.shape[0], self.N), dtype, self.device, stream)
        with torch.cuda.device(self.device):
            _lib.moe_w4a4_linear_bf16(x, self.weight, out, bias=self.bias, function=self.function, gated=self.gated,
                                      row_scale=row_scale, addend=addend, stream=stream)
        return out


class Bf16MLP:
    """Two Bf16Linears in a row, a shared expert's: a (gated) one with its function, and
    the down projection.  What is between them is rounded to bfloat16."""

    def __init__(self, gate_up: Bf16Linear, down: Bf16Linear):
        if gate_up.N != down.K or gate_up.device != down.device:
            raise ValueError(f"down: from {down.K} on {down.device}, expected {gate_up.N} on {gate_up.device}")
        self.gate_up, self.down, self.K, self.N, self.device = gate_up, down, gate_up.K, down.N, down.device

    def _held(self):
        return self.down._held()

    def forward(self, x, out=None, addend=None, row_scale=None, dtype=torch.bfloat16, stream=None):
        """x bf16 [T, K] -> out [T, N], the rest for the down projection (Bf16Linear.forward)."""
        h = self.gate_up.forward(x, stream=stream)
        return self.down.forward(h, out=out, addend=addend, row_scale=row_scale, dtype=dtype, stream=stream)


class Bf16Experts(_Block):
    """Routed experts with bfloat16 weights (moe_w4a4_experts_bf16), for expert layers left
    unquantized: forward and forward_block as MoeW4A4Layer's.  Holds the weights and a
    workspace for max_tokens tokens; calls that may run at the same time need
    Bf16Experts of their own (with_capacity)."""
    mma_type = _lib.MOE_MMA_MXF4_X_MXF4      # (of codes that nothing asks for)

    def __init__(self, w1, w2, topk: int, max_tokens: int, function: int = _lib.MOE_FN_SILU):
        """w1 bf16 [E, 2I, H] (gate rows, then up rows), w2 bf16 [E, H, I]."""
        if w1.dim() != 3 or w2.dim() != 3:
            raise ValueError(f"w1 {tuple(w1.shape)} and w2 {tuple(w2.shape)}: expected [E, 2I, H] and [E, H, I]")
        self.E, self.H, self.I = w2.shape
        self.k, self.max_tokens, self.device = topk, max_tokens, _gpu(w1.device)
        for name, w, shape in (("w1", w1, (self.E, 2 * self.I, self.H)), ("w2", w2, (self.E, self.H, self.I))):
            if _lib._fits(w, name, (torch.bfloat16,), shape, self.device.index) % 16:
                raise ValueError(f"{name}: not 16-byte aligned")
        self.cfg = _lib.make_experts_bf16_cfg(self.H, self.I, self.E, topk, max_tokens, function)
        self.w1, self.w2 = w1, w2
        self.workspace = torch.empty(_lib.moe_w4a4_experts_bf16_query(self.cfg), dtype=torch.uint8, device=self.device)

    def with_capacity(self, max_tokens: int) -> "Bf16Experts":
        """The same weights with a workspace of their own."""
        return Bf16Experts(self.w1, self.w2, self.k, max_tokens, self.cfg.function)

    def forward(self, x, topk_ids, topk_weights, out=None, stream=None):
        """x bf16 [T, H]; topk_ids int32 [T, k] (ids outside [0, E) are skipped);
        topk_weights float32 [T, k]; out bf16 [T, H] or None (may be x)."""
        if out is None:
            out = _output((x.shape[0], self.H), torch.bfloat16, self.device, stream)
        with torch.cuda.device(self.device):
            _lib.moe_w4a4_experts_bf16(self.cfg, self.w1, self.w2, x, topk_ids, topk_weights, out, self.workspace,
                                       stream=stream)
        return out

    # ---- the steps of forward_block ------------------------------------------
    def _held(self):
        return self.w1, self.w2, self.workspace

    def _experts(self, T, y, codes, ids, weights, out) -> None:
        _lib.moe_w4a4_experts_bf16(self.cfg, self.w1, self.w2, y, ids, weights, out, self.workspace)
