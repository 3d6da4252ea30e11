"""GPU tier: the bfloat16 operators at the ends of what they take and on the paths that small sizes
do not reach.  Whole numbers that bfloat16 holds where a comparison is exact."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from block_scaled_fp4_pre_amd.layer import Bf16Experts
from tests.gpu_support import log

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def whole(g, most, *shape):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(BF)


@pytest.mark.parametrize("T", [(1 << 23) + 5, 1 << 24])
def test_experts_of_the_most_tokens(T):
    """relu(x g^T) (x u^T) with one-hot gate rows is at most 8, y at most 64, weights are powers of two."""
    log(f"[test] experts_bf16 {T} tokens")
    H = I = 8
    g = torch.Generator(device="cuda").manual_seed(1)
    eye = torch.eye(8, device="cuda").to(BF)
    w1 = torch.cat([eye.expand(2, 8, 8), whole(g, 1, 2, 8, 8)], 1).contiguous()
    w2 = whole(g, 1, 2, 8, 8)
    x = whole(g, 1, T, H)
    ids = torch.randint(-1, 3, (T, 1), generator=g, device="cuda").to(torch.int32)          # -1 and 2: no expert
    wt = torch.exp2(torch.randint(-1, 2, (T, 1), generator=g, device="cuda").float())
    layer = Bf16Experts(w1, w2, 1, T, _lib.MOE_FN_RELU)
    out = torch.full((T, H), 77.0, dtype=BF, device="cuda")
    layer.forward(x, ids, wt, out=out)
    torch.cuda.synchronize()
    want = torch.zeros((T, H), device="cuda")
    for e in (0, 1):
        h = torch.relu(x.float()) * (x.float() @ w1[e, 8:].float().t().contiguous())
        want += torch.where(ids == e, wt * (h @ w2[e].float().t().contiguous()), 0.0)
    assert torch.equal(out.float(), want)
