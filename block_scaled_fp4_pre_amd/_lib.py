"""ctypes binding of libmoe_w4a4.so (C ABI in include/moe_w4a4.h).

Argument marshalling only: tensors are passed as raw device pointers, the
current torch stream as the HIP stream, and status codes become MoeError.
Every step of the layer runs in the library's HIP kernels; if the library is
missing this module raises at import time -- there is no other code path.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_w4a4.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_ECAPACITY, MOE_EWORKSPACE, MOE_ENODEVICE, MOE_EHIP, MOE_ESCRATCH = range(8)
MOE_NOALLOC_SCRATCH_BYTES = 64 << 20
MOE_MMA_MXF4_X_MXF4, MOE_MMA_FP8_X_MXF4, MOE_MMA_NVF4_X_NVF4 = 0, 1, 2
MOE_ACT_SWIGLU = 0
MOE_STAGE_QUANT, MOE_STAGE_ROUTE, MOE_STAGE_GEMM1, MOE_STAGE_GEMM2, MOE_STAGE_COMBINE = 1, 2, 4, 8, 16
MOE_STAGE_ALL = 31
MOE_MEGA_MAX_ROWS = 256          # routed rows the single-launch forward takes
MOE_MEGA_AUTO_ROWS = 48          # routed rows up to which moe_w4a4_forward takes it (MXFP4)
MOE_MEGA_AUTO_ROWS_FP8 = 24      # the same for fp8xfp4
MOE_MEGA_STATE_BYTES = 144 << 10  # its workspace state region (offset 0), zero before its first call
MOE_MEGA_ERR_WORD = 800           # uint64 word of that region that a wait which gave up sets
MOE_MEGA_HCOUNT_WORD = 816        # first per-expert h count of that region (words hcount + e)

MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID, MOE_SCORE_SQRTSOFTPLUS = 0, 1, 2

# Every symbol include/moe_w4a4.h declares.
EXPORTED = (
    "moe_w4a4_query",
    "moe_w4a4_quantize",
    "moe_w4a4_quantize_nvfp4",
    "moe_w4a4_prepare_weights",
    "moe_w4a4_prepare_weights_nvfp4",
    "moe_w4a4_forward",
    "moe_w4a4_forward_mega",
    "moe_w4a4_forward_noalloc",
    "moe_w4a4_status_string",
    "moe_w4a4_workspace_layout",
    "moe_w4a4_run_stages",
    "moe_w4a4_add_rmsnorm",
    "moe_w4a4_router",
    "moe_w4a4_linear_query",
    "moe_w4a4_linear_prepare",
    "moe_w4a4_linear",
)


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


class moe_w4a4_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "hidden", "inter", "num_experts", "topk", "max_tokens", "group_size", "mma_type", "activation")]


class moe_w4a4_linear_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("in_features", "out_features", "max_tokens", "mma_type")]


class moe_w4a4_ws_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in (
        "xq", "xsf", "counts", "offsets", "sorted_rows", "pos", "hist", "hq", "hsf", "y", "tiles",
        "num_tiles", "xsf_planes", "mega", "total")]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                      "(python block_scaled_fp4_pre_amd/build.py)")
# torch ships its own HIP runtime.  Loading torch first makes the library bind
# to that same runtime (same devices, streams and allocations); loading the
# library first would bring in a second runtime next to torch's.
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_sz = ctypes.c_size_t
_i32 = ctypes.c_int32
_CFG = ctypes.POINTER(moe_w4a4_cfg)
_lib.moe_w4a4_query.argtypes = [_CFG, ctypes.POINTER(_sz), ctypes.POINTER(_sz)]
_lib.moe_w4a4_quantize.argtypes = [_i32, _P, ctypes.c_int64, _i32, _P, _P, _P]
_lib.moe_w4a4_quantize_nvfp4.argtypes = [_i32, _P, ctypes.c_int64, _i32, ctypes.c_float, _P, _P, _P]
_lib.moe_w4a4_prepare_weights.argtypes = [_CFG, _P, _P, _P, _P, _P, _sz, _P]
_lib.moe_w4a4_prepare_weights_nvfp4.argtypes = [_CFG, _P, _P, _P, _P, _P, _P, ctypes.c_float, ctypes.c_float, _P,
                                                _sz, _P]
_lib.moe_w4a4_forward.argtypes = [_CFG, _P, _i32, _P, _P, _P, _P, _P, _sz, _P]
_lib.moe_w4a4_forward_mega.argtypes = [_CFG, _P, _i32, _P, _P, _P, _P, _P, _sz, _P]
_lib.moe_w4a4_forward_noalloc.argtypes = [_CFG, _P, _i32, _P, _P, _P, _P, _P]
_lib.moe_w4a4_status_string.argtypes = [ctypes.c_int]
_lib.moe_w4a4_status_string.restype = ctypes.c_char_p
_lib.moe_w4a4_workspace_layout.argtypes = [_CFG, ctypes.POINTER(moe_w4a4_ws_layout)]
_lib.moe_w4a4_run_stages.argtypes = [_CFG, _P, _i32, _P, _P, _P, _P, _P, _sz, ctypes.c_uint32, _P, _P]
_f32, _i64 = ctypes.c_float, ctypes.c_int64
_LCFG = ctypes.POINTER(moe_w4a4_linear_cfg)
_lib.moe_w4a4_add_rmsnorm.argtypes = [_i32, _i32, _i32, _i64, _i32, _P, _P, _P, _f32, _f32, _P, _P, _P, _P, _P]
_lib.moe_w4a4_router.argtypes = [_i32, _i32, _i64, _i32, _i32, _i32, _i32, _P, _P, _i32, _f32, _P, _P, _P]
_lib.moe_w4a4_linear_query.argtypes = [_LCFG, ctypes.POINTER(_sz), ctypes.POINTER(_sz)]
_lib.moe_w4a4_linear_prepare.argtypes = [_LCFG, _P, _P, _P, _sz, _P]
_lib.moe_w4a4_linear.argtypes = [_LCFG, _P, _i32, _P, _P, _P, _P, _i32, _P, _P, _sz, _P]
for _n in EXPORTED:
    if _n != "moe_w4a4_status_string":
        getattr(_lib, _n).restype = ctypes.c_int


def lib() -> ctypes.CDLL:
    return _lib


def status_string(status: int) -> str:
    return _lib.moe_w4a4_status_string(int(status)).decode()


def _check(st: int, where: str) -> None:
    if st != MOE_OK:
        raise MoeError(st, where)


def _ptr(t) -> int | None:
    """Device address of a tensor (None -> NULL); no copies, no conversions."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


_BF16_LIKE = ("bfloat16", "int16", "uint16")   # bf16 values or their bit patterns


def _expect(t, name: str, dtypes, shape=None, min_rows=None) -> None:
    """Raise ValueError unless tensor t (if given) has one of the dtypes (by
    name), the exact shape (None entries match any size) or at least min_rows
    rows, and lives on the current device.  The library sees only pointers:
    a wrong dtype or a short buffer would be read or written out of bounds
    by the kernels, so it is refused here."""
    if t is None or isinstance(t, int):
        return
    dt = str(t.dtype).replace("torch.", "")
    if dt not in dtypes:
        raise ValueError(f"{name}: dtype {dt}, expected {' or '.join(dtypes)}")
    if shape is not None:
        if t.dim() != len(shape) or any(w is not None and w != g for g, w in zip(t.shape, shape)):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected "
                             f"({', '.join('*' if w is None else str(w) for w in shape)})")
        if min_rows is not None and t.shape[0] < min_rows:
            raise ValueError(f"{name}: {t.shape[0]} rows, at least {min_rows} needed")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a device tensor, got one on {t.device}")
    import torch
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _check_forward_tensors(cfg, num_tokens, x, topk_ids, topk_weights, out, workspace, prepared,
                           gemm1_acc=None) -> None:
    T, H, k, I = int(num_tokens), cfg.hidden, cfg.topk, cfg.inter
    _expect(x, "x", _BF16_LIKE, (None, H), T)
    _expect(topk_ids, "topk_ids", ("int32",), (None, k), T)
    _expect(topk_weights, "topk_weights", ("float32",), (None, k), T)
    _expect(out, "out", _BF16_LIKE, (None, H), T)
    _expect(workspace, "workspace", ("uint8",))
    _expect(prepared, "prepared", ("uint8",))
    _expect(gemm1_acc, "gemm1_acc", ("float32",), (None, 2 * I), T * k)


def _stream(stream) -> int | None:
    if stream is not None:
        return int(stream)
    import torch
    return torch.cuda.current_stream().cuda_stream


def make_cfg(hidden: int, inter: int, num_experts: int, topk: int, max_tokens: int,
             group_size: int | None = None, mma_type: int = MOE_MMA_MXF4_X_MXF4,
             activation: int = MOE_ACT_SWIGLU) -> moe_w4a4_cfg:
    """group_size None: the MMA type's own (16 for NVFP4, else 32)."""
    if group_size is None:
        group_size = 16 if mma_type == MOE_MMA_NVF4_X_NVF4 else 32
    return moe_w4a4_cfg(hidden, inter, num_experts, topk, max_tokens, group_size, mma_type, activation)


def scale_group(cfg) -> int:
    """Elements per scale byte of cfg's MMA type."""
    return 16 if cfg.mma_type == MOE_MMA_NVF4_X_NVF4 else 32


def moe_w4a4_query(cfg: moe_w4a4_cfg):
    """(prepared_bytes, workspace_bytes)."""
    p, w = _sz(), _sz()
    _check(_lib.moe_w4a4_query(ctypes.byref(cfg), ctypes.byref(p), ctypes.byref(w)), "moe_w4a4_query")
    return p.value, w.value


def moe_w4a4_workspace_layout(cfg: moe_w4a4_cfg) -> dict:
    lay = moe_w4a4_ws_layout()
    _check(_lib.moe_w4a4_workspace_layout(ctypes.byref(cfg), ctypes.byref(lay)), "moe_w4a4_workspace_layout")
    return {n: getattr(lay, n) for n, _ in moe_w4a4_ws_layout._fields_}


def moe_w4a4_quantize(src, codes, scales, stream=None) -> None:
    """src: device bf16 (or uint16 bit patterns) / float32 [rows, cols];
    codes uint8 [rows, cols/2]; scales uint8 [rows, cols/32]."""
    import torch
    if src.dtype in (torch.bfloat16, torch.uint16, torch.int16):
        dt = 0
    elif src.dtype == torch.float32:
        dt = 1
    else:
        raise ValueError(f"unsupported dtype {src.dtype}")
    if src.dim() != 2:
        raise ValueError(f"src: expected [rows, cols], got shape {tuple(src.shape)}")
    rows, cols = src.shape
    _expect(src, "src", ("bfloat16", "int16", "uint16", "float32"))
    _expect(codes, "codes", ("uint8",), (rows, cols // 2))
    _expect(scales, "scales", ("uint8",), (rows, cols // 32))
    _check(_lib.moe_w4a4_quantize(dt, _ptr(src), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_w4a4_quantize")


def moe_w4a4_quantize_nvfp4(src, g: float, codes, scales, stream=None) -> None:
    """NVFP4 with tensor scale g: src device bf16 (or uint16 bit patterns) /
    float32 [rows, cols]; codes uint8 [rows, cols/2]; scales uint8 [rows, cols/16]."""
    import torch
    if src.dtype in (torch.bfloat16, torch.uint16, torch.int16):
        dt = 0
    elif src.dtype == torch.float32:
        dt = 1
    else:
        raise ValueError(f"unsupported dtype {src.dtype}")
    if src.dim() != 2:
        raise ValueError(f"src: expected [rows, cols], got shape {tuple(src.shape)}")
    rows, cols = src.shape
    _expect(src, "src", ("bfloat16", "int16", "uint16", "float32"))
    _expect(codes, "codes", ("uint8",), (rows, cols // 2))
    _expect(scales, "scales", ("uint8",), (rows, cols // 16))
    _check(_lib.moe_w4a4_quantize_nvfp4(dt, _ptr(src), rows, cols, float(g), _ptr(codes), _ptr(scales),
                                        _stream(stream)), "moe_w4a4_quantize_nvfp4")


def moe_w4a4_prepare_weights_nvfp4(cfg, w1_codes, w1_scales, w1_tensor_scales, w2_codes, w2_scales,
                                   w2_tensor_scales, x_tensor_scale: float, h_tensor_scale: float, prepared,
                                   stream=None) -> None:
    E, H, I = cfg.num_experts, cfg.hidden, cfg.inter
    _expect(w1_codes, "w1_codes", ("uint8",), (E, 2 * I, H // 2))
    _expect(w1_scales, "w1_scales", ("uint8",), (E, 2 * I, H // 16))
    _expect(w1_tensor_scales, "w1_tensor_scales", ("float32",), (E,))
    _expect(w2_codes, "w2_codes", ("uint8",), (E, H, I // 2))
    _expect(w2_scales, "w2_scales", ("uint8",), (E, H, I // 16))
    _expect(w2_tensor_scales, "w2_tensor_scales", ("float32",), (E,))
    _expect(prepared, "prepared", ("uint8",))
    _check(_lib.moe_w4a4_prepare_weights_nvfp4(
        ctypes.byref(cfg), _ptr(w1_codes), _ptr(w1_scales), _ptr(w1_tensor_scales), _ptr(w2_codes), _ptr(w2_scales),
        _ptr(w2_tensor_scales), float(x_tensor_scale), float(h_tensor_scale), _ptr(prepared),
        prepared.numel() * prepared.element_size(), _stream(stream)), "moe_w4a4_prepare_weights_nvfp4")


def moe_w4a4_prepare_weights(cfg, w1_codes, w1_scales, w2_codes, w2_scales, prepared, stream=None) -> None:
    E, H, I = cfg.num_experts, cfg.hidden, cfg.inter
    _expect(w1_codes, "w1_codes", ("uint8",), (E, 2 * I, H // 2))
    _expect(w1_scales, "w1_scales", ("uint8",), (E, 2 * I, H // 32))
    _expect(w2_codes, "w2_codes", ("uint8",), (E, H, I // 2))
    _expect(w2_scales, "w2_scales", ("uint8",), (E, H, I // 32))
    _expect(prepared, "prepared", ("uint8",))
    _check(_lib.moe_w4a4_prepare_weights(ctypes.byref(cfg), _ptr(w1_codes), _ptr(w1_scales), _ptr(w2_codes),
                                         _ptr(w2_scales), _ptr(prepared), prepared.numel() * prepared.element_size(),
                                         _stream(stream)), "moe_w4a4_prepare_weights")


def moe_w4a4_forward(cfg, prepared, num_tokens: int, x, topk_ids, topk_weights, out, workspace,
                     stream=None) -> None:
    """x bf16 [>= T, H], topk_ids int32 [>= T, k], topk_weights float32
    [>= T, k], out bf16 [>= T, H], all on the current device; T = num_tokens."""
    _check_forward_tensors(cfg, num_tokens, x, topk_ids, topk_weights, out, workspace, prepared)
    _check(_lib.moe_w4a4_forward(ctypes.byref(cfg), _ptr(prepared), int(num_tokens), _ptr(x), _ptr(topk_ids),
                                 _ptr(topk_weights), _ptr(out), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_w4a4_forward")


def moe_w4a4_forward_mega(cfg, prepared, num_tokens: int, x, topk_ids, topk_weights, out, workspace,
                          stream=None) -> None:
    """The forward as one kernel launch (decode sizes); arguments as moe_w4a4_forward."""
    _check_forward_tensors(cfg, num_tokens, x, topk_ids, topk_weights, out, workspace, prepared)
    _check(_lib.moe_w4a4_forward_mega(ctypes.byref(cfg), _ptr(prepared), int(num_tokens), _ptr(x), _ptr(topk_ids),
                                      _ptr(topk_weights), _ptr(out), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_w4a4_forward_mega")


def moe_w4a4_forward_noalloc(cfg, prepared, num_tokens: int, x, topk_ids, topk_weights, out,
                             stream=None) -> None:
    """The forward on the library's static scratch instead of a workspace."""
    _check_forward_tensors(cfg, num_tokens, x, topk_ids, topk_weights, out, None, prepared)
    _check(_lib.moe_w4a4_forward_noalloc(ctypes.byref(cfg), _ptr(prepared), int(num_tokens), _ptr(x),
                                         _ptr(topk_ids), _ptr(topk_weights), _ptr(out), _stream(stream)),
           "moe_w4a4_forward_noalloc")


def moe_w4a4_run_stages(cfg, prepared, num_tokens: int, x, topk_ids, topk_weights, out, workspace,
                        stages: int, gemm1_acc=None, stream=None) -> None:
    _check_forward_tensors(cfg, num_tokens, x, topk_ids, topk_weights, out, workspace, prepared, gemm1_acc)
    _check(_lib.moe_w4a4_run_stages(ctypes.byref(cfg), _ptr(prepared), int(num_tokens), _ptr(x), _ptr(topk_ids),
                                    _ptr(topk_weights), _ptr(out), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), int(stages), _ptr(gemm1_acc),
                                    _stream(stream)), "moe_w4a4_run_stages")


# ---- operators around the layer ----------------------------------------------
# These calls are a few microseconds of GPU work, so their checks go straight to
# the tensors' properties; the rules are _expect's.

def _raw_stream(stream, device_index: int) -> int:
    return int(stream) if stream is not None else torch._C._cuda_getCurrentRawStream(device_index)


def _fits(t, name: str, dtypes, shape, device_index: int, contiguous: bool = True) -> int:
    """Device address of a (contiguous) tensor of one of the dtypes, of that
    shape, on device `device_index`; else ValueError."""
    if t.dtype in dtypes and t.shape == shape and t.get_device() == device_index and (t.is_contiguous() or not contiguous):
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a device tensor, got one on {t.device}")
    if t.device.index != device_index:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{device_index}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


_BF16 = (torch.bfloat16,)
_BF16_F32 = (torch.bfloat16, torch.float32)
_U8, _F32, _I32 = (torch.uint8,), (torch.float32,), (torch.int32,)


def _device_of(t, name: str) -> int:
    """Index of the current device, on which t has to be."""
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a device tensor, got one on {t.device}")
    return torch._C._cuda_getDevice()      # (t exists, so the runtime is initialised)


def moe_w4a4_add_rmsnorm(x, residual, weight, eps: float, residual_out=None, y=None, codes=None, scales=None,
                         mma_type: int = MOE_MMA_MXF4_X_MXF4, tensor_scale: float = 1.0, stream=None) -> None:
    """h = x + residual (or x), into residual_out; y = h * weight / rms(h) in
    bf16; codes and scales = y quantized as mma_type's activations (NVFP4 under
    tensor_scale).  x bf16 [rows, cols]; residual None, or bf16 / float32 [rows,
    cols]; weight bf16 / float32 [cols]; residual_out like residual (may be it;
    None exactly when residual is None); y None or bf16 [rows, cols] (may be x);
    codes and scales both None, or uint8 [rows, cols/2] (E4M3: cols) and
    [rows, cols/32] (NVFP4: cols/16)."""
    dev = _device_of(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x: expected [rows, cols], got shape {tuple(x.shape)}")
    rows, cols = shape = x.shape
    px = _fits(x, "x", _BF16, shape, dev)
    pw = _fits(weight, "weight", _BF16_F32, (cols,), dev)
    pr = pro = py = pc = ps = None
    res_dtype = 0
    if residual is not None:
        pr = _fits(residual, "residual", _BF16_F32, shape, dev)
        if residual_out is None:
            raise ValueError("residual_out: needed with a residual")
        pro = _fits(residual_out, "residual_out", (residual.dtype,), shape, dev)
        res_dtype = 1 if residual.dtype is torch.float32 else 0
    elif residual_out is not None:
        raise ValueError("residual_out: given without a residual")
    if y is not None:
        py = _fits(y, "y", _BF16, shape, dev)
    if codes is not None or scales is not None:
        if codes is None or scales is None:
            raise ValueError("codes and scales go together")
        pc = _fits(codes, "codes", _U8, (rows, cols if mma_type == MOE_MMA_FP8_X_MXF4 else cols // 2), dev)
        ps = _fits(scales, "scales", _U8, (rows, cols // (16 if mma_type == MOE_MMA_NVF4_X_NVF4 else 32)), dev)
    st = _lib.moe_w4a4_add_rmsnorm(mma_type, res_dtype, 1 if weight.dtype is torch.float32 else 0, rows, cols, px, pr,
                                   pw, eps, tensor_scale, pro, py, pc, ps, _raw_stream(stream, dev))
    if st != MOE_OK:
        raise MoeError(st, "moe_w4a4_add_rmsnorm")


def moe_w4a4_router(logits, topk_ids, topk_weights, bias=None, scoring: int = MOE_SCORE_SOFTMAX, num_groups: int = 1,
                    topk_groups: int = 1, renormalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """Experts and weights of every token from the router's logits: logits bf16
    / float32 [T, E]; bias None or float32 [E] (added to the scores for the
    choice only); topk_ids int32 [T, k] and topk_weights float32 [T, k] are
    written (k is their width), ready for a forward."""
    dev = _device_of(logits, "logits")
    if logits.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError(f"logits {tuple(logits.shape)} and topk_ids {tuple(topk_ids.shape)}: expected [T, E] and [T, k]")
    T, E = logits.shape
    k = topk_ids.shape[1]
    pl = _fits(logits, "logits", _BF16_F32, (T, E), dev)
    pi = _fits(topk_ids, "topk_ids", _I32, (T, k), dev)
    pw = _fits(topk_weights, "topk_weights", _F32, (T, k), dev)
    pb = None if bias is None else _fits(bias, "bias", _F32, (E,), dev)
    st = _lib.moe_w4a4_router(1 if logits.dtype is torch.float32 else 0, scoring, T, E, k, num_groups, topk_groups, pl,
                              pb, 1 if renormalize else 0, scale, pi, pw, _raw_stream(stream, dev))
    if st != MOE_OK:
        raise MoeError(st, "moe_w4a4_router")


def _check_router_config(num_experts: int, topk: int, scoring: int, num_groups: int, topk_groups: int,
                         scale: float) -> None:
    """Raise what moe_w4a4_router would raise for its plain arguments (the library
    checks them for no tokens too)."""
    _check(_lib.moe_w4a4_router(1, scoring, 0, num_experts, topk, num_groups, topk_groups, None, None, 1, scale, None,
                                None, None), "moe_w4a4_router")


def make_linear_cfg(in_features: int, out_features: int, max_tokens: int,
                    mma_type: int = MOE_MMA_MXF4_X_MXF4) -> moe_w4a4_linear_cfg:
    return moe_w4a4_linear_cfg(in_features, out_features, max_tokens, mma_type)


def moe_w4a4_linear_query(cfg: moe_w4a4_linear_cfg):
    """(prepared_bytes, workspace_bytes)."""
    p, w = _sz(), _sz()
    _check(_lib.moe_w4a4_linear_query(ctypes.byref(cfg), ctypes.byref(p), ctypes.byref(w)), "moe_w4a4_linear_query")
    return p.value, w.value


def moe_w4a4_linear_prepare(cfg: moe_w4a4_linear_cfg, codes, scales, prepared, stream=None) -> None:
    """codes uint8 [N, K/2], scales uint8 [N, K/32]: canonical MXFP4 weights."""
    dev = _device_of(codes, "codes")
    N, K = cfg.out_features, cfg.in_features
    pc = _fits(codes, "codes", _U8, (N, K // 2), dev)
    ps = _fits(scales, "scales", _U8, (N, K // 32), dev)
    pw = _fits(prepared, "prepared", _U8, prepared.shape, dev)
    _check(_lib.moe_w4a4_linear_prepare(ctypes.byref(cfg), pc, ps, pw, prepared.numel(), _raw_stream(stream, dev)),
           "moe_w4a4_linear_prepare")


def moe_w4a4_linear(cfg: moe_w4a4_linear_cfg, prepared, x, out, workspace, xq=None, xsf=None, addend=None,
                    stream=None) -> None:
    """out [T, N] (bf16 or float32) = Q(x) W^T (+ addend bf16 [T, N]); x bf16
    [T, K], or None and xq uint8 [T, K/2] (E4M3: [T, K]) with xsf uint8 [T, K/32]."""
    dev = _device_of(out, "out")
    pw = _fits(prepared, "prepared", _U8, prepared.shape, dev)
    pk = _fits(workspace, "workspace", _U8, workspace.shape, dev)
    _linear_call(ctypes.byref(cfg), cfg.in_features, cfg.out_features, cfg.mma_type, dev, pw, x, out, pk,
                 workspace.numel(), xq, xsf, addend, stream, prepared.numel())


def _linear_call(cfg_ref, K: int, N: int, mma_type: int, dev: int, prepared: int, x, out, workspace: int,
                 workspace_bytes: int, xq, xsf, addend, stream, prepared_bytes: int | None = None) -> None:
    """moe_w4a4_linear with the caller's own buffers as addresses
    (layer.W4A4Linear, which made its weights' buffer: prepared_bytes None)."""
    px = pq = ps = pa = None
    if x is not None:
        if xq is not None or xsf is not None:
            raise ValueError("x: given together with xq or xsf")
        T = x.shape[0] if x.dim() == 2 else -1
        px = _fits(x, "x", _BF16, (T, K), dev)
    else:
        if xq is None or xsf is None:
            raise ValueError("either x, or xq and xsf")
        T = xq.shape[0] if xq.dim() == 2 else -1
        pq = _fits(xq, "xq", _U8, (T, K if mma_type == MOE_MMA_FP8_X_MXF4 else K // 2), dev)
        ps = _fits(xsf, "xsf", _U8, (T, K // 32), dev)
    if addend is not None:
        pa = _fits(addend, "addend", _BF16, (T, N), dev)
    po = _fits(out, "out", _BF16_F32, (T, N), dev)
    if prepared_bytes is not None:
        need = _sz()
        _check(_lib.moe_w4a4_linear_query(cfg_ref, ctypes.byref(need), None), "moe_w4a4_linear_query")
        if prepared_bytes < need.value:
            raise ValueError(f"prepared: {prepared_bytes} bytes, at least {need.value} needed")
    st = _lib.moe_w4a4_linear(cfg_ref, prepared, T, px, pq, ps, pa, 1 if out.dtype is torch.float32 else 0, po,
                              workspace, workspace_bytes, _raw_stream(stream, dev))
    if st != MOE_OK:
        raise MoeError(st, "moe_w4a4_linear")
