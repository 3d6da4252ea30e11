"""GPU tier: moe_w4a4_post_norm where a workgroup takes several rows (more than 512 of more than
8192 values), and rows past the registers in place; tolerances as in tests/test_gpu_post_norm.py."""
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from tests.gpu_support import log
from tests.test_gpu_post_norm import EPS, FP8, MX4, NV4, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,res_f32,gate,mma", [
    (1030, 8224, False, "row", FP8), (520, 8224, True, "full", None), (1030, 16384, False, "channel", NV4),
    (520, 16384, True, None, MX4), (1030, 16416, False, "row", FP8), (520, 16416, True, "full", NV4)])
def test_several_rows_a_workgroup(rows, cols, res_f32, gate, mma):
    log(f"[test] post_norm rows {rows} cols {cols} residual f32 {res_f32}")
    check(rows, cols, 7, res_f32, gate=gate, mma=mma)


@pytest.mark.parametrize("rows,cols", [(520, 8224), (33, 16416), (520, 16416), (3, 65536)])
@pytest.mark.parametrize("res_f32", [False, True])
def test_in_place(rows, cols, res_f32):
    log(f"[test] post_norm in place, rows {rows} cols {cols} residual f32 {res_f32}")
    check(rows, cols, 8, res_f32, gate="channel", mma=FP8, inplace=True)


@pytest.mark.parametrize("rows,cols", [(1030, 8224), (1030, 16416), (5, 65536)])
@pytest.mark.parametrize("post", [False, True])
def test_y_in_the_place_of_the_residual_and_h_in_the_place_of_x(rows, cols, post):
    """The bits of the call with outputs of their own, and those of its rows in calls of 100."""
    log(f"[test] post_norm other places, rows {rows} cols {cols} post {post}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, r = (torch.randn((rows, cols), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.randn(cols, generator=g, device="cuda").to(torch.bfloat16)
    kw = dict(post_weight=w if post else None, scale=0.6, next_weight=w)
    h, y = torch.empty_like(x), torch.empty_like(x)
    _lib.moe_w4a4_post_norm(x, r, h, EPS, y=y, **kw)
    parts = [torch.empty_like(x) for _ in range(2)]
    for a in range(0, rows, 100):
        s = slice(a, a + 100)
        _lib.moe_w4a4_post_norm(x[s], r[s], parts[0][s], EPS, y=parts[1][s], **kw)
    x2, r2 = x.clone(), r.clone()
    _lib.moe_w4a4_post_norm(x2, r2, x2, EPS, y=r2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(x2, h) and torch.equal(r2, y) and torch.equal(parts[0], h) and torch.equal(parts[1], y)
