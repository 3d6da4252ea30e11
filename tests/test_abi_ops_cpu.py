"""Refusals of the operators around the layer (norm, router, linear), with no
GPU: the library's host checks under sanitizers (tests/ops_host_check.cpp), the
C entry points themselves, and the binding's checks of tensors."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from block_scaled_fp4_pre_amd import _lib

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "block_scaled_fp4_pre_amd", "csrc")
FAKE = ctypes.c_void_p(1 << 20)            # aligned, never dereferenced


def test_every_check_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "ops_host_check"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "validate.cpp"), os.path.join(HERE, "ops_host_check.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ)
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith(" 0 failed"), r.stdout + r.stderr


def test_entry_points_run_the_checks_before_any_hip_call():
    L = _lib.lib()
    far = [ctypes.c_void_p((2 + i) << 20) for i in range(3)]
    norm = lambda rows, cols=64, x=FAKE: L.moe_w4a4_add_rmsnorm(1, 0, 0, rows, cols, x, None, FAKE, 1e-6, 1.0, None,  # noqa: E731
                                                                 far[0], far[1], far[2], None)
    assert norm(4, 40) == _lib.MOE_EUNSUPPORTED and norm(4, 64, None) == _lib.MOE_EINVAL and norm(0) == _lib.MOE_OK
    router = lambda T, E=64: L.moe_w4a4_router(1, 0, T, E, 6, 1, 1, FAKE, None, 1, 1.0, FAKE, FAKE, None)  # noqa: E731
    assert router(4, 600) == _lib.MOE_EUNSUPPORTED and router(-1) == _lib.MOE_EINVAL and router(0) == _lib.MOE_OK
    cfg = _lib.make_linear_cfg(64, 32, 8)
    pb, wb = _lib.moe_w4a4_linear_query(cfg)
    lin = lambda T, ws=wb: L.moe_w4a4_linear(ctypes.byref(cfg), FAKE, T, FAKE, None, None, None, 0, far[0], FAKE, ws, None)  # noqa: E731
    assert lin(9) == _lib.MOE_ECAPACITY and lin(4, wb - 1) == _lib.MOE_EWORKSPACE and lin(0, 0) == _lib.MOE_OK
    assert L.moe_w4a4_linear_prepare(ctypes.byref(cfg), FAKE, FAKE, FAKE, pb - 1, None) == _lib.MOE_EWORKSPACE
    if not torch.cuda.is_available():
        assert norm(4) == router(4) == lin(4) == _lib.MOE_ENODEVICE
        assert L.moe_w4a4_linear_prepare(ctypes.byref(cfg), FAKE, FAKE, FAKE, pb, None) == _lib.MOE_ENODEVICE
    with pytest.raises(_lib.MoeError) as ei:
        _lib.moe_w4a4_linear_query(_lib.make_linear_cfg(64, 32, 8, _lib.MOE_MMA_NVF4_X_NVF4))
    assert ei.value.status == _lib.MOE_EUNSUPPORTED


class Cuda(torch.Tensor):
    """A host tensor that says it is on cuda:0, for the checks ahead of the library."""
    is_cuda = True
    device = torch.device("cuda", 0)


def _t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Cuda)


@pytest.fixture
def current_device_0(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(_lib, "_raw_stream", lambda stream, dev: None)
    monkeypatch.setattr(_lib, "_lib", None)                 # the library must not be reached


BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.mark.parametrize("change", [
    dict(x=_t((4, 64), F32)), dict(x=_t((256,))), dict(weight=_t((63,))), dict(weight=_t((64,), torch.float16)),
    dict(residual=_t((4, 32))), dict(residual=_t((4, 64), torch.float16)), dict(residual_out=None),
    dict(residual=None), dict(residual_out=_t((4, 64), F32)), dict(y=_t((3, 64))), dict(y=_t((4, 64), F32)),
    dict(codes=None), dict(scales=None), dict(codes=_t((4, 32), U8)), dict(scales=_t((4, 4), U8)),
    dict(x=_t((64, 4)).t()), dict(x=torch.zeros((4, 64), dtype=BF)), dict(y=torch.zeros((4, 64), dtype=BF)),
    dict(mma_type=_lib.MOE_MMA_MXF4_X_MXF4), dict(mma_type=_lib.MOE_MMA_NVF4_X_NVF4)], ids=lambda c: ",".join(c))
def test_norm_binding_refuses(current_device_0, change):
    a = dict(x=_t((4, 64)), residual=_t((4, 64)), weight=_t((64,), F32), eps=1e-6, residual_out=_t((4, 64)),
             y=_t((4, 64)), codes=_t((4, 64), U8), scales=_t((4, 2), U8), mma_type=_lib.MOE_MMA_FP8_X_MXF4)
    with pytest.raises(ValueError):
        _lib.moe_w4a4_add_rmsnorm(**{**a, **change})


@pytest.mark.parametrize("change", [
    dict(logits=_t((4, 64), torch.float16)), dict(logits=_t((256,), F32)), dict(topk_ids=_t((4, 6), torch.int64)),
    dict(topk_ids=_t((3, 6), I32)), dict(topk_ids=_t((4,), I32)), dict(topk_weights=_t((4, 5), F32)),
    dict(topk_weights=_t((4, 6))), dict(bias=_t((63,), F32)), dict(bias=_t((64,))),
    dict(logits=torch.zeros((4, 64)))], ids=lambda c: ",".join(c))
def test_router_binding_refuses(current_device_0, change):
    a = dict(logits=_t((4, 64), F32), topk_ids=_t((4, 6), I32), topk_weights=_t((4, 6), F32), bias=_t((64,), F32))
    with pytest.raises(ValueError):
        _lib.moe_w4a4_router(**{**a, **change})


@pytest.mark.parametrize("change", [
    dict(x=_t((4, 96))), dict(x=_t((4, 64), F32)), dict(x=_t((256,))), dict(x=None), dict(xq=_t((4, 32), U8)),
    dict(x=None, xq=_t((4, 64), U8), xsf=_t((4, 2), U8)), dict(x=None, xq=_t((4, 32), U8), xsf=_t((4, 3), U8)),
    dict(x=None, xq=_t((4, 32), U8)), dict(out=_t((3, 32))), dict(out=_t((4, 32), torch.float16)),
    dict(addend=_t((4, 32), F32)), dict(addend=_t((4, 31))), dict(workspace=_t((64,), F32)),
    dict(prepared=torch.zeros(64, dtype=U8))], ids=lambda c: ",".join(c))
def test_linear_binding_refuses(current_device_0, change):
    cfg = _lib.make_linear_cfg(64, 32, 8)
    a = dict(cfg=cfg, prepared=_t((1 << 16,), U8), x=_t((4, 64)), out=_t((4, 32)), workspace=_t((1 << 16,), U8))
    with pytest.raises(ValueError):
        _lib.moe_w4a4_linear(**{**a, **change})


def test_binding_refuses_another_device(current_device_0, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="current device"):
        _lib.moe_w4a4_router(_t((4, 64), F32), _t((4, 6), I32), _t((4, 6), F32))


@pytest.mark.parametrize("operator", ["norm", "linear"])
def test_buffers_that_share_an_address(operator, tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "ops_overlap_check"
    cmd = [gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "validate.cpp"), os.path.join(HERE, "ops_overlap_check.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe), operator], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith(" 0 failed"), r.stdout + r.stderr


def test_binding_refuses_weights_that_are_too_short(monkeypatch):
    """The product reads all of the prepared weights, and is told only where they begin."""
    def reached(*a):
        raise AssertionError("the library was called")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(_lib, "_raw_stream", lambda stream, dev: None)
    monkeypatch.setattr(_lib._lib, "moe_w4a4_linear", reached)
    cfg = _lib.make_linear_cfg(64, 32, 8)
    pb, wb = _lib.moe_w4a4_linear_query(cfg)
    call = lambda n: _lib.moe_w4a4_linear(cfg, _t((n,), U8), _t((4, 64)), _t((4, 32)), _t((wb,), U8))  # noqa: E731
    with pytest.raises(ValueError, match="prepared"):
        call(pb - 1)
    with pytest.raises(AssertionError, match="library"):
        call(pb)


def test_linear_refuses_shared_weights_with_gaps():
    """A strided view has enough elements, but not from its first address on."""
    from block_scaled_fp4_pre_amd.layer import W4A4Linear
    pb, _ = _lib.moe_w4a4_linear_query(_lib.make_linear_cfg(64, 32, 8))
    for bad in (_t((2 * pb,), U8)[::2], _t((pb - 1,), U8), _t((1,), U8).expand(pb)):
        with pytest.raises(ValueError, match="prepared"):
            W4A4Linear(64, 32, 8, "cuda:0", prepared=bad)


def _block_layer():
    from block_scaled_fp4_pre_amd.layer import MoeW4A4Layer
    layer = MoeW4A4Layer.__new__(MoeW4A4Layer)
    layer.H, layer.I, layer.E, layer.k, layer.max_tokens = 64, 64, 16, 3, 8
    layer.mma_type, layer.device = _lib.MOE_MMA_MXF4_X_MXF4, torch.device("cuda", 0)
    return layer


def _block_linear(K, N, max_tokens, index=0):
    from block_scaled_fp4_pre_amd.layer import W4A4Linear
    lin = W4A4Linear.__new__(W4A4Linear)
    lin.K, lin.N, lin.max_tokens, lin.device = K, N, max_tokens, torch.device("cuda", index)
    return lin


# what a step behind the norm would refuse
BLOCK_REFUSALS = [
    dict(gate_weight=_t((16, 64), F32)), dict(gate_weight=_t((15, 64))), dict(gate_weight=_t((16, 32))),
    dict(gate_weight=torch.zeros((16, 64), dtype=BF)), dict(gate_weight=_block_linear(64, 16, 3)),
    dict(gate_weight=_block_linear(64, 17, 8)), dict(gate_weight=_block_linear(64, 16, 8, 1)),
    dict(bias=_t((15,), F32)), dict(bias=_t((16,))), dict(scoring=3), dict(num_groups=5), dict(num_groups=4, topk_groups=5),
    dict(num_groups=8, topk_groups=1), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(shared=_block_linear(64, 64, 3)), dict(shared=_block_linear(64, 32, 8)), dict(shared=_block_linear(32, 64, 8)),
    dict(shared=_block_linear(64, 64, 8, 1)), dict(shared=_t((64, 64))), dict(out=_t((4, 32))), dict(out=_t((3, 64))),
    dict(out=_t((4, 64), F32)), dict(out=_t((64, 4)).t()), dict(out=_t((5, 64)), shared=_block_linear(64, 64, 8)),
    dict(out=_t((1, 257))[:, 1:].reshape(4, 64))]


@pytest.mark.parametrize("change", BLOCK_REFUSALS, ids=lambda c: ",".join(f"{k}{i}" for i, k in enumerate(c)))
def test_block_refuses_before_the_norm(monkeypatch, change):
    def reached(*a, **k):
        raise AssertionError("the norm was called")
    monkeypatch.setattr(_lib, "moe_w4a4_add_rmsnorm", reached)
    a = dict(x=_t((4, 64)), residual=_t((4, 64)), norm_weight=_t((64,), F32), eps=1e-6, gate_weight=_t((16, 64)))
    with pytest.raises((ValueError, _lib.MoeError)):
        _block_layer().forward_block(**{**a, **change})


def test_block_refuses_an_output_in_the_place_of_the_residual():
    a = dict(x=_t((4, 64)), norm_weight=_t((64,), F32), eps=1e-6, gate_weight=_t((16, 64)))
    r = _t((4, 64))
    with pytest.raises(ValueError, match="residual_out"):
        _block_layer().forward_block(residual=r, residual_out=r, out=r, **a)
    with pytest.raises(ValueError, match="holds"):
        _block_layer().forward_block(residual=None, **{**a, "x": _t((9, 64))})
