"""forward_block's refusals of what its later steps would refuse, before the norm may have
overwritten x and the residual (no GPU: tensors that say they are on one)."""
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from block_scaled_fp4_pre_amd.layer import Bf16Linear, Bf16MLP
from tests.test_abi_bf16_cpu import BLOCK, _experts_layer
from tests.test_abi_ops_cpu import _block_layer, _block_linear, _t, current_device_0  # noqa: F401

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def experts_layer():
    layer = _experts_layer()
    layer.w1, layer.w2, layer.workspace = _t((16, 128, 64)), _t((16, 64, 64)), _t((1 << 12,), U8)
    return layer


@pytest.fixture
def no_norm(monkeypatch):
    def reached(*a, **k):
        raise AssertionError("the norm was called")
    monkeypatch.setattr(_lib, "moe_w4a4_add_rmsnorm", reached)


def first(t, shape, dtype=None):
    """The first values of t's memory as a tensor of that shape."""
    n = 1
    for s in shape:
        n *= s
    return (t if dtype is None else t.view(dtype)).reshape(-1)[:n].view(shape)


@pytest.mark.parametrize("make", [_block_layer, experts_layer], ids=["w4a4", "bf16"])
@pytest.mark.parametrize("place", ["out", "residual_out"])
@pytest.mark.parametrize("name", ["post_weight", "next_weight"])
def test_a_weight_of_the_norm_behind_in_the_place_of_an_output(no_norm, make, place, name):
    t = _t((4, 64))
    with pytest.raises(ValueError, match=name):
        make().forward_block(**BLOCK, **{place: t, name: first(t, (64,))})


def test_out_in_the_place_of_weights(no_norm):
    down = Bf16Linear(_t((64, 128)), bias=_t((64 * 64,), F32)[:64])
    layer = experts_layer()
    packed = _block_linear(64, 64, 8)
    packed.prepared, packed.workspace = _t((1 << 12,), U8), _t((1 << 12,), U8)
    for lay, shared, t in ((layer, None, layer.w1), (layer, None, layer.w2), (layer, None, layer.workspace.view(BF)),
                           (_block_layer(), down_of(down), down.weight), (_block_layer(), down_of(down), down.bias.view(BF)),
                           (_block_layer(), packed, packed.prepared.view(BF)), (layer, packed, packed.workspace.view(BF))):
        out = torch.as_strided(t, (4, 64), (64, 1)) if t.numel() < 256 else first(t, (4, 64))
        with pytest.raises(ValueError, match="place of weights"):
            lay.forward_block(**BLOCK, shared=shared, out=out)


def down_of(down):
    return Bf16MLP(Bf16Linear(_t((256, 64)), gated=True), down)


def test_more_tokens_than_the_shared_mlp_takes(no_norm):
    """2^36 values between its two products at most: 2^20 tokens of 65536."""
    layer, T = experts_layer(), (1 << 20) + 1
    layer.max_tokens = 1 << 21
    mlp = Bf16MLP(Bf16Linear(_t((1 << 16, 64))), Bf16Linear(_t((64, 1 << 16))))
    x = _t((T, 64))
    args = {**BLOCK, "x": x, "residual": x}
    with pytest.raises(ValueError, match=f"takes {1 << 20} tokens"):
        layer.forward_block(**args, shared=mlp)
