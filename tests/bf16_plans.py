"""A ragged size for every kernel that the bfloat16 linears' rule can choose
(csrc/launch_bf16.h), for every way of calling it: (kernel, gated, groups, T, K, N), groups 0 for
a dense product.  K ends inside a step of 64, N inside a vector and a tile, T inside a
tile.  tests/test_bf16_plans.py holds that each size takes the kernel of its row and
that no other kernel is reached; tests/test_gpu_bf16_plans.py runs them."""
import math

import numpy as np

# in the order of enum Bf16Plan
PLANS = ("split 16x8", "split 16x8 wide", "split 16x16", "split 16x32", "split 32x32", "split 32x64", "split 16x8 once",
         "split 32x16 once", "split 32x32 once", "tile 64x64", "tile 128x64", "tile 128x128", "tile 256x128", "tile 256x256",
         "tile 128x64 once", "tile 256x128 once")

CASES = [
    ("split 16x8", False, 0, 7, 456, 3301), ("split 16x8", True, 0, 5, 456, 1709),
    ("split 16x8", False, 3, 4, 456, 3301), ("split 16x8", True, 3, 3, 456, 1709),
    ("split 16x8 wide", False, 0, 5, 712, 131), ("split 16x8 wide", True, 0, 3, 712, 77),
    ("split 16x8 wide", False, 5, 23, 712, 131), ("split 16x8 wide", True, 5, 21, 712, 77),
    ("split 16x16", False, 0, 169, 456, 213), ("split 16x16", True, 0, 241, 456, 73),
    ("split 16x16", False, 3, 403, 456, 81), ("split 16x16", True, 3, 405, 456, 41),
    ("split 16x32", False, 0, 385, 456, 257), ("split 16x32", True, 0, 307, 456, 161),
    ("split 16x32", False, 3, 463, 456, 211), ("split 16x32", True, 3, 647, 456, 73),
    ("split 32x32", False, 0, 225, 456, 659), ("split 32x32", True, 0, 353, 456, 217),
    ("split 32x32", False, 3, 735, 456, 209), ("split 32x32", True, 3, 637, 456, 121),
    ("split 32x64", False, 0, 649, 456, 579), ("split 32x64", True, 0, 483, 456, 385),
    ("split 32x64", False, 3, 883, 456, 417), ("split 32x64", True, 3, 1563, 456, 113),
    ("split 16x8 once", False, 0, 7, 4168, 16289), ("split 16x8 once", True, 0, 5, 4168, 8089),
    ("split 16x8 once", False, 8, 13, 2088, 4019), ("split 16x8 once", True, 8, 15, 712, 5891),
    ("split 32x16 once", False, 0, 13, 4168, 16131), ("split 32x16 once", True, 0, 11, 2088, 16079),
    ("split 32x16 once", False, 12, 67, 2088, 2681), ("split 32x16 once", True, 5, 29, 2088, 3219),
    ("split 32x32 once", False, 0, 27, 4168, 16163), ("split 32x32 once", True, 0, 21, 4168, 8059),
    ("split 32x32 once", False, 8, 101, 2088, 4023), ("split 32x32 once", True, 3, 43, 2088, 5373),
    ("tile 64x64", False, 0, 323, 456, 1365), ("tile 64x64", True, 0, 261, 456, 817),
    ("tile 64x64", False, 5, 1103, 456, 385), ("tile 64x64", True, 3, 1083, 456, 209),
    ("tile 128x64", False, 0, 2917, 456, 449), ("tile 128x64", True, 0, 1409, 456, 483),
    ("tile 128x64", False, 3, 3839, 456, 323), ("tile 128x64", True, 3, 2907, 456, 225),
    ("tile 128x128", False, 0, 769, 456, 3337), ("tile 128x128", True, 0, 1153, 456, 1133),
    ("tile 128x128", False, 3, 3881, 456, 645), ("tile 128x128", True, 3, 7277, 456, 161),
    ("tile 256x128", False, 0, 5525, 456, 705), ("tile 256x128", True, 0, 1601, 456, 1255),
    ("tile 256x128", False, 3, 9491, 456, 385), ("tile 256x128", True, 3, 3615, 456, 551),
    ("tile 256x256", False, 0, 27475, 456, 257), ("tile 256x256", True, 0, 27785, 456, 129),
    ("tile 256x256", False, 12, 27097, 456, 265), ("tile 256x256", True, 8, 27051, 456, 129),
    ("tile 128x64 once", False, 8, 145, 2088, 4031), ("tile 128x64 once", True, 12, 251, 712, 3931),
    ("tile 256x128 once", False, 5, 249, 2088, 6439), ("tile 256x128 once", True, 8, 467, 2088, 2023),
]
IDS = [f"{plan} {'gated' if gated else 'plain'} {'groups' if groups else 'dense'}".replace(" ", "_")
       for plan, gated, groups, *_ in CASES]


def offsets(T, groups):
    """Bounds of uneven groups of T rows in all: one holds half of them, one is empty."""
    rng = np.random.default_rng([T, groups])
    share = rng.random(groups) + 0.2
    share[groups // 2], share[groups - 1] = share.sum(), 0.0
    bounds = np.round(T * np.concatenate([[0], np.cumsum(share)]) / share.sum()).astype(np.int32)
    assert bounds[-1] == T and bounds[-2] == T
    return bounds


# Whole operands up to `largest(K)`: no part of a sum of K products passes 2^24, so that every
# sum is exact in float32 in any order, and float32 is needed for it.
def largest(K):
    return min(127, math.isqrt(2 ** 24 // K))


def whole(rng, shape, most):
    return rng.integers(-most, most + 1, size=shape)
