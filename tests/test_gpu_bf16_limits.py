"""GPU tier: the bfloat16 operators at the ends of what they take and on the paths that small sizes
do not reach.  Whole numbers that bfloat16 holds where a comparison is exact."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from block_scaled_fp4_pre_amd.layer import Bf16Experts
from tests.bf16_plans import CASES
from tests.gpu_support import log
from tests.test_gpu_bf16_plans import Product

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


@pytest.mark.parametrize("case", [c for c in CASES if c[0] in ("split 32x64", "tile 64x64", "tile 256x128", "tile 256x256") and c[2]],
                         ids=lambda c: f"{c[0]} {'gated' if c[1] else 'plain'}".replace(" ", "_"))
def test_gathered_rows_past_2_gib(case):
    """Rows of x more than 2^31 bytes behind its first (which lies as far into its buffer), for
    kernels of many rows: the same number for number as from the rows brought together."""
    log(f"[test] grouped_bf16 far gathered rows {case}")
    p = Product(case, 1, seed=4)
    stride, Tx = 4096, 500000                                # 4.1 GB, below 2^31 elements
    buf = torch.full((300000 + Tx, stride), float("nan"), dtype=BF, device="cuda")
    far = buf[300000:, :p.K]
    at = torch.from_numpy(p.rng.choice(Tx, size=p.T, replace=False).astype(np.int32))
    at[0], at[p.T - 1] = Tx - 1, 262144                      # the last row, and the first past 2 GiB
    at = at.cuda()
    near = p.x
    far[at.long()] = near
    near = far[at.long()].contiguous()                       # (a row drawn twice holds the later one's values)
    p.x = near
    want = p.run(torch.float32)
    p.x, p.rows, p.gather = far, at, 1
    got = p.run(torch.float32)
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())
