"""GPU tier: moe_w4a4_experts_bf16 is its steps: with one expert a token and a weight of 1 the
combine rounds nothing, and the outputs are the bits of the two grouped products called one by
one; with every function, against the fp64 oracle too (the layer's parity bar, as in
tests/test_gpu_bf16_linear.py)."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_pre_amd import _lib
from block_scaled_fp4_pre_amd.layer import Bf16Experts
from oracle import bf16_linear
from oracle.route import route
from tests.gpu_support import dev, dev_bf16, log
from tests.test_gpu_bf16_linear import FN, rows_like, values, weights

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# (one block routes up to 8192 rows, several those of the last size)
@pytest.mark.parametrize("T,H,I,E", [(1, 64, 40, 4), (33, 256, 128, 8), (700, 72, 200, 12), (9000, 64, 72, 5)])
@pytest.mark.parametrize("fn", bf16_linear.FUNCTIONS)
def test_the_bits_of_the_steps(T, H, I, E, fn):
    log(f"[test] experts_bf16 {fn} T {T} H {H} I {I} E {E}, one expert a token")
    rng = np.random.default_rng([T, H, FN[fn]])
    (w1b, w1), (w2b, w2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
    layer = Bf16Experts(dev_bf16(w1b), dev_bf16(w2b), 1, T, FN[fn])
    layer.workspace.fill_(0xA5)
    xb, x = rows_like(rng, T, H)
    ids, ones = rng.integers(0, E, size=(T, 1)).astype(np.int32), np.ones((T, 1), np.float32)
    if T > 5:
        ids[2], ids[4] = -1, E
    xd = dev_bf16(xb)
    out = layer.forward(xd, dev(ids), dev(ones))
    _, offsets, order, pos = route(ids, E)
    rows = torch.zeros(T, dtype=torch.int32, device="cuda")
    rows[:len(order)] = dev(order)
    h, y = torch.empty((T, I), dtype=BF, device="cuda"), torch.zeros((T, H), dtype=BF, device="cuda")
    _lib.moe_w4a4_grouped_linear_bf16(xd, layer.w1, dev(offsets), h, rows=rows, function=FN[fn], gated=True)
    _lib.moe_w4a4_grouped_linear_bf16(h, layer.w2, dev(offsets), y)
    torch.cuda.synchronize()
    at = torch.from_numpy(np.asarray(pos, np.int64).reshape(-1)).cuda()
    want = torch.where((at >= 0)[:, None], y[at.clamp(min=0)], torch.zeros((), dtype=BF, device="cuda"))
    assert torch.equal(out, want)
    ref = bf16_linear.experts(x, ids, ones, w1, w2, fn)
    assert np.linalg.norm(values(out) - ref) <= 5e-3 * np.linalg.norm(ref)
