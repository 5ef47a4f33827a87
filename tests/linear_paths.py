"""Which way a dense product takes (moed_selftest_linear), and sizes that between them take every one of them."""
import math
import random

import torch

from output_centric_expert_amd import moedecode as md

PAIRS = [(x, w) for x in ("bf16", "f32") for w in ("bf16", "f32")]
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# The last ways of a product that the sizes of test_gpu_block.py leave out: the largest bfloat16 tile with k split (its
# parts begin at even and odd steps and end inside K or not), one to three steps of every tile, every tile with whole
# steps and K even and odd, few outputs of many rows.
MORE_SIZES = [
    (2048, 7168, 2304), (5997, 4610, 260), (6534, 7443, 140), (4000, 4096, 24), (2, 8960, 2), (3, 2, 2), (3, 8960, 2),
    (196, 2, 320), (202, 1024, 1384), (215, 68, 306), (215, 69, 292), (226, 704, 807), (262, 128, 706), (264, 130, 6819),
    (276, 96, 3271), (293, 32, 685), (322, 1152, 581), (323, 896, 660), (328, 67, 5414), (338, 1, 178), (387, 192, 495),
    (389, 66, 505), (393, 131, 512), (449, 2, 129), (483, 64, 386), (517, 128, 7359), (588, 2, 6577), (805, 96, 5019),
    (811, 138, 227), (1097, 192, 3616), (1129, 131, 3591), (1173, 32, 3472), (1521, 66, 1317), (1811, 954, 129),
    (1861, 6720, 129), (2153, 1024, 68), (2188, 5079, 1032), (2265, 71, 3681), (2384, 64, 1665), (2415, 65, 392),
    (3283, 256, 1153), (3321, 134, 1248), (3343, 67, 1201), (3830, 130, 2190), (3844, 128, 2049), (4163, 4288, 131),
    (5037, 141, 1538), (5447, 137, 295), (5468, 6386, 270), (5475, 4160, 263), (5483, 2798, 138), (5495, 128, 270),
    (5520, 64, 261), (5531, 3178, 187), (5577, 192, 267), (5591, 256, 270), (5788, 3264, 144), (5943, 4441, 145),
    (6563, 64, 1156), (6588, 66, 1294), (6684, 2, 1167), (6752, 1456, 27), (7244, 193, 514), (7390, 192, 1035)]


def way(B, K, N, x, w):
    """What makes one run of the kernels differ from another: kernel, tile, side, k split or not, rows that begin at dwords or
    not, how K ends (in whole steps, behind some, in the first); of tiles the steps too: up to three that fill the
    buffers, or with k split whether a part begins at an odd one."""
    kernel, shape, swapped, splits, step, part = md.moed_selftest_linear(B, K, N, TYPES[x], TYPES[w])
    if kernel == 0:
        return x, w, kernel
    end = "whole" if K % step == 0 else "behind" if K > step else "inside"
    dwords = x == w == "f32" or K % 2 == 0
    steps = (K + step - 1) // step
    pipeline = None if kernel == 1 else min(steps, 4) if splits == 1 else "odd" if part % 2 else "even"
    return x, w, kernel, shape, swapped, splits > 1, dwords, end, pipeline


def reachable(count=200000, products=2.0 ** 35):
    """The ways of random sizes of up to 8192 rows and outputs and 32768 values of k, and a size for each."""
    rng = random.Random(1)
    rows = lambda most: int(math.exp(rng.uniform(0, math.log(most))))  # noqa: E731
    ways = {}
    for _ in range(count):
        B, K, N = rows(8192) + 1, rows(32768), rows(8192) + 1
        r = rng.random()
        K = max(64, K // 64 * 64) if r < 0.4 else K // 2 * 2 + 2 if r < 0.6 else K
        if B * K * N <= products:
            for pair in PAIRS:
                ways.setdefault(way(B, K, N, *pair), (B, K, N))
    return ways
