"""Refusals of the bfloat16 operators (linear, grouped linear, experts, norm after a
block), with no GPU: the library's host checks under sanitizers
(tests/bf16_host_check.cpp), the C entry points themselves, and the binding's checks
of tensors."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from tests.test_abi_ops_cpu import CSRC, HERE, ROOT, Cuda, _block_layer, _block_linear, _t, current_device_0  # noqa: F401

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def test_every_check_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "bf16_host_check"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "validate.cpp"), os.path.join(CSRC, "validate_bf16.cpp"),
           os.path.join(HERE, "bf16_host_check.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ)
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith(" 0 failed"), r.stdout + r.stderr


def test_entry_points_run_the_checks_before_any_hip_call():
    L = _lib.lib()
    at = [ctypes.c_void_p((1 + i) << 20) for i in range(8)]
    lin = lambda T, K=64: L.moe_w4a4_linear_bf16(T, K, 32, at[0], K, at[1], 0, 0, 0, None, None, 0, None, 0, 0, at[2],  # noqa: E731
                                                 32, None)
    grp = lambda R, E=4: L.moe_w4a4_grouped_linear_bf16(E, R, 64, 32, at[3], at[0], R, 64, None, 1, at[1], 0, 0, 0,  # noqa: E731
                                                        None, None, 0, None, 0, 0, at[2], 32, None)
    post = lambda rows, cols=64: L.moe_w4a4_post_norm(0, 0, 0, 0, 0, rows, cols, at[0], at[1], None, None, 1.0, None,  # noqa: E731
                                                      1e-6, 1.0, at[2], None, None, None, None)
    cfg = _lib.make_experts_bf16_cfg(64, 32, 8, 2, 16)
    wb = _lib.moe_w4a4_experts_bf16_query(cfg)
    exp = lambda T, ws=wb: L.moe_w4a4_experts_bf16(ctypes.byref(cfg), at[0], at[1], T, at[2], at[3], at[4], at[5], at[6],  # noqa: E731
                                                   ws, None)
    assert lin(4, 60) == _lib.MOE_EUNSUPPORTED and lin(-1) == _lib.MOE_EINVAL and lin(0) == _lib.MOE_OK
    assert grp(4, 513) == _lib.MOE_EUNSUPPORTED and grp(-1) == _lib.MOE_EINVAL and grp(0) == _lib.MOE_OK
    assert post(4, 40) == _lib.MOE_EUNSUPPORTED and post(-1) == _lib.MOE_EINVAL and post(0) == _lib.MOE_OK
    assert exp(17) == _lib.MOE_ECAPACITY and exp(4, wb - 1) == _lib.MOE_EWORKSPACE and exp(0) == _lib.MOE_OK
    if not torch.cuda.is_available():
        assert lin(4) == grp(4) == post(4) == exp(4) == _lib.MOE_ENODEVICE
    with pytest.raises(_lib.MoeError) as ei:
        _lib.moe_w4a4_experts_bf16_query(_lib.make_experts_bf16_cfg(60, 32, 8, 2, 16))
    assert ei.value.status == _lib.MOE_EUNSUPPORTED


def test_workspace_layout():
    """Regions in order, 256-byte aligned, none short."""
    cfg = _lib.make_experts_bf16_cfg(64, 40, 8, 3, 1000)
    R = 3000
    up = lambda b: (b + 255) // 256 * 256                                            # noqa: E731
    want = sum(map(up, (8 * 4, 9 * 4, R * 4, R * 4, 3 * 8 * 4, R * 40 * 2, R * 64 * 2)))
    assert _lib.moe_w4a4_experts_bf16_query(cfg) == want


# (`_lib._lib` is None there: a call that passes the binding's checks ends in AttributeError)
@pytest.mark.parametrize("change", [
    dict(x=_t((4, 64), F32)), dict(x=_t((256,))), dict(x=_t((3, 64))), dict(x=_t((64, 4)).t()),
    dict(x=_t((1, 64)).expand(4, 64)), dict(x=_t((4, 128))[:, ::2]), dict(x=_t((8, 32)).as_strided((4, 64), (32, 1))),
    dict(x=torch.zeros((4, 64), dtype=BF)), dict(weight=_t((63, 64))), dict(weight=_t((32, 64))), dict(weight=_t((64, 64), F32)),
    dict(weight=_t((64, 128))[:, :64]), dict(out=_t((4, 32), torch.float16)), dict(out=_t((5, 32))), dict(out=_t((128,))),
    dict(out=_t((32, 4)).t()), dict(out=_t((4, 1)).expand(4, 32)), dict(bias=_t((32,))), dict(bias=_t((64,), torch.float16)),
    dict(bias=_t((128,))[::2]), dict(row_scale=_t((4,))), dict(row_scale=_t((4, 1), F32)), dict(row_scale=_t((1,), F32).expand(4)),
    dict(addend=_t((4, 31))), dict(addend=_t((4, 32), torch.float16)), dict(addend=_t((1, 32)).expand(4, 32)),
    dict(addend=torch.zeros((4, 32), dtype=BF))], ids=lambda c: ",".join(c))
def test_linear_binding_refuses(current_device_0, change):  # noqa: F811
    a = dict(x=_t((4, 64)), weight=_t((64, 64)), out=_t((4, 32)), bias=_t((64,), F32), gated=True, row_scale=_t((4,), F32),
             addend=_t((4, 32)))
    with pytest.raises(AttributeError):
        _lib.moe_w4a4_linear_bf16(**a)
    with pytest.raises(ValueError):
        _lib.moe_w4a4_linear_bf16(**{**a, **change})


@pytest.mark.parametrize("change", [
    dict(x=_t((4, 32))), dict(x=_t((4, 64), F32)), dict(x=_t((256,))), dict(weight=_t((3, 32, 32))), dict(weight=_t((32, 64))),
    dict(weight=_t((2, 32, 64))), dict(offsets=_t((3,), I32)), dict(offsets=_t((4,), torch.int64)),
    dict(offsets=torch.zeros(4, dtype=I32)), dict(rows=_t((5,), I32)), dict(rows=_t((6,), torch.int64)), dict(out=_t((6, 31))),
    dict(out=_t((7, 32))), dict(bias=_t((32,))), dict(bias=_t((3, 31))), dict(row_scale=_t((5,), F32)),
    dict(addend=_t((5, 32)))], ids=lambda c: ",".join(c))
def test_grouped_binding_refuses(current_device_0, change):  # noqa: F811
    a = dict(x=_t((4, 64)), weight=_t((3, 32, 64)), offsets=_t((4,), I32), out=_t((6, 32)), rows=_t((6,), I32), row_divisor=2,
             bias=_t((3, 32)), row_scale=_t((6,), F32), addend=_t((6, 32), F32))
    with pytest.raises(AttributeError):
        _lib.moe_w4a4_grouped_linear_bf16(**a)
    with pytest.raises(ValueError):
        _lib.moe_w4a4_grouped_linear_bf16(**{**a, **change})


@pytest.mark.parametrize("change", [
    dict(w1=_t((8, 64, 32))), dict(w2=_t((8, 64, 64))), dict(w2=_t((7, 64, 32))), dict(x=_t((4, 32))), dict(x=_t((64,))),
    dict(topk_ids=_t((4, 2), torch.int64)), dict(topk_ids=_t((3, 2), I32)), dict(topk_weights=_t((4, 2))),
    dict(out=_t((5, 64))), dict(out=_t((4, 64), F32)), dict(workspace=_t((64,), F32))], ids=lambda c: ",".join(c))
def test_experts_binding_refuses(current_device_0, change):  # noqa: F811
    a = dict(cfg=_lib.make_experts_bf16_cfg(64, 32, 8, 2, 16), w1=_t((8, 64, 64)), w2=_t((8, 64, 32)), x=_t((4, 64)),
             topk_ids=_t((4, 2), I32), topk_weights=_t((4, 2), F32), out=_t((4, 64)), workspace=_t((1 << 16,), U8))
    with pytest.raises(AttributeError):
        _lib.moe_w4a4_experts_bf16(**a)
    with pytest.raises(ValueError):
        _lib.moe_w4a4_experts_bf16(**{**a, **change})


@pytest.mark.parametrize("change", [
    dict(x=_t((4, 64), F32)), dict(x=_t((256,))), dict(x=_t((64, 4)).t()), dict(residual=_t((4, 32))),
    dict(residual=_t((4, 64), torch.float16)), dict(residual_out=_t((4, 64), F32)), dict(residual_out=_t((3, 64))),
    dict(post_weight=_t((63,))), dict(post_weight=_t((64,), F32)), dict(next_weight=_t((64,), torch.float16)),
    dict(gate=_t((63,))), dict(gate=_t((1, 64))), dict(gate=_t((4, 2))), dict(gate=_t((3, 1))), dict(gate=_t((4, 64), torch.float16)),
    dict(gate=_t((4, 1, 1))), dict(gate=_t(())), dict(gate=_t((4, 1)).expand(4, 64)), dict(y=_t((4, 64), F32)), dict(y=_t((5, 64))),
    dict(codes=None), dict(scales=None), dict(codes=_t((4, 32), U8)), dict(scales=_t((4, 4), U8)),
    dict(mma_type=_lib.MOE_MMA_MXF4_X_MXF4)], ids=lambda c: ",".join(c))
def test_post_norm_binding_refuses(current_device_0, change):  # noqa: F811
    a = dict(x=_t((4, 64)), residual=_t((4, 64)), residual_out=_t((4, 64)), eps=1e-6, post_weight=_t((64,)), gate=_t((4, 1), F32),
             next_weight=_t((64,)), y=_t((4, 64)), codes=_t((4, 64), U8), scales=_t((4, 2), U8),
             mma_type=_lib.MOE_MMA_FP8_X_MXF4)
    with pytest.raises(AttributeError):
        _lib.moe_w4a4_post_norm(**a)
    with pytest.raises(ValueError):
        _lib.moe_w4a4_post_norm(**{**a, **change})


def test_bindings_refuse_another_device(current_device_0, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="current device"):
        _lib.moe_w4a4_linear_bf16(_t((4, 64)), _t((32, 64)), _t((4, 32)))
    with pytest.raises(ValueError, match="current device"):
        _lib.moe_w4a4_post_norm(_t((4, 64)), _t((4, 64)), _t((4, 64)), 1e-6)


def test_a_single_rows_stride_says_nothing():
    """A row alone may have any stride, a column too; what the library is told fits both."""
    one = _t((1, 64)).as_strided((1, 64), (3, 1))
    assert _lib._rows_of(one, "x", (BF,), (1, 64), 0) == (one.data_ptr(), 64)
    wide = _t((4, 72))
    assert _lib._rows_of(wide[:, 8:], "x", (BF,), (4, 64), 0) == (wide.data_ptr() + 16, 72)
    assert _lib._rows_of(_t((4, 3))[:, :1], "x", (BF,), (4, 1), 0)[1] == 3


# ---- the objects ---------------------------------------------------------------
def _linear16(K, N, index=0):
    from block_scaled_fp4_pre_amd.layer import Bf16Linear
    lin = Bf16Linear.__new__(Bf16Linear)
    lin.K, lin.N, lin.device = K, N, torch.device("cuda", index)
    return lin


def test_objects_refuse():
    from block_scaled_fp4_pre_amd.layer import Bf16Experts, Bf16Linear, Bf16MLP
    for bad in (torch.zeros((32, 64), dtype=BF), _t((32, 64), F32), _t((64,)), _t((64, 32)).t(), _t((1, 32 * 64 + 1))[:, 1:].reshape(32, 64)):
        with pytest.raises(ValueError):
            Bf16Linear(bad)
    with pytest.raises(_lib.MoeError):
        Bf16Linear(_t((32, 60)))
    with pytest.raises(_lib.MoeError):
        Bf16Linear(_t((32, 64)), function=9)
    with pytest.raises(ValueError):
        Bf16Linear(_t((33, 64)), gated=True)
    with pytest.raises(ValueError):
        Bf16Linear(_t((32, 64)), bias=_t((16,)))
    assert Bf16Linear(_t((32, 64)), gated=True).N == 16
    for down in (_linear16(31, 64), _linear16(32, 64, 1)):
        with pytest.raises(ValueError):
            Bf16MLP(_linear16(64, 32), down)
    for w1, w2 in ((_t((4, 64, 64)), _t((4, 64, 16))), (_t((64, 64)), _t((4, 64, 32))), (_t((4, 64, 64)), _t((3, 64, 32))),
                   (_t((4, 64, 64), F32), _t((4, 64, 32)))):
        with pytest.raises(ValueError):
            Bf16Experts(w1, w2, 2, 8)


BLOCK = dict(x=_t((4, 64)), residual=_t((4, 64)), norm_weight=_t((64,), F32), eps=1e-6, gate_weight=_t((16, 64)))


def _experts_layer():
    from block_scaled_fp4_pre_amd.layer import Bf16Experts
    layer = Bf16Experts.__new__(Bf16Experts)
    layer.H, layer.I, layer.E, layer.k, layer.max_tokens, layer.device = 64, 64, 16, 3, 8, torch.device("cuda", 0)
    return layer


@pytest.mark.parametrize("make", [_block_layer, _experts_layer], ids=["w4a4", "bf16"])
@pytest.mark.parametrize("change", [
    dict(gate_weight=_linear16(64, 17)), dict(gate_weight=_linear16(32, 16)), dict(gate_weight=_linear16(64, 16, 1)),
    dict(shared=_linear16(64, 32)), dict(shared=_linear16(64, 64, 1)), dict(shared=_block_linear(64, 64, 3)),
    dict(shared=_t((64, 64))), dict(post_weight=_t((63,))), dict(post_weight=_t((64,), torch.float16)),
    dict(post_weight=_t((64,)), next_weight=_t((64,), F32)), dict(next_weight=_t((64,), torch.float16)),
    dict(post_gate=_t((4, 2))), dict(post_gate=_t((3, 1))), dict(post_gate=_t(())), dict(post_gate=_t((1, 65))[:, 1:].reshape(64)[:64].view(64)[1:]),
    dict(post_gate=_t((4, 64), torch.float16)), dict(post_scale=float("inf")), dict(post_scale=float("nan")),
    dict(post_scale=1.0, out=_t((5, 64))), dict(post_scale=1.0, out=_t((4, 64), torch.int16)),
    dict(x=_t((9, 64)), residual=_t((9, 64)))], ids=lambda c: ",".join(f"{k}{i}" for i, k in enumerate(c)))
def test_block_refuses_before_the_norm(monkeypatch, make, change):
    def reached(*a, **k):
        raise AssertionError("the norm was called")
    monkeypatch.setattr(_lib, "moe_w4a4_add_rmsnorm", reached)
    with pytest.raises(ValueError):
        make().forward_block(**{**BLOCK, **change})


def test_block_with_a_norm_behind_refuses_outputs_in_the_place_of_what_it_reads():
    x, g = _t((4, 64)), _t((4, 64))
    with pytest.raises(ValueError, match="place of x"):
        _block_layer().forward_block(**{**BLOCK, "x": x, "residual": None}, out=x, post_scale=1.0)
    with pytest.raises(ValueError, match="post_gate"):
        _block_layer().forward_block(**BLOCK, out=g, post_gate=g)
