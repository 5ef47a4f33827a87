"""The GPU tests of moe_linear run every way that a product can take: a choice by other sizes or costs, or a kernel more, has
to come with sizes here (no GPU needed; nothing is launched)."""
import ctypes

import pytest

from linear_paths import MORE_SIZES, PAIRS, reachable, way
from output_centric_expert_amd import moedecode as md
from test_abi import lib  # noqa: F401
from test_gpu_block import SIZES


def test_every_way_is_tested(lib):  # noqa: F811
    tested = {way(*size, *pair) for size in SIZES + MORE_SIZES for pair in PAIRS}
    missing = {w: size for w, size in reachable().items() if w not in tested}
    assert not missing, missing


def test_ways_of_known_products(lib):  # noqa: F811
    assert md.moed_selftest_linear(1, 4096, 4096) == (0, 0, 0, 1, 0, 0)
    kernel, shape, swapped, splits, step, _ = md.moed_selftest_linear(4000, 4096, 24)
    assert (kernel, shape, swapped, splits, step) == (1, 2, 1, 1, 64)
    kernel, shape, _, splits, step, part = md.moed_selftest_linear(2048, 7168, 2304)
    assert (kernel, shape, step) == (2, 0, 64) and splits > 1 and (splits - 1) * part < 112 <= splits * part


def test_way_refusals(lib):  # noqa: F811
    path = (ctypes.c_int32 * 6)()
    for size in ((0, 64, 64), (-1, 64, 64), (1 << 22, 64, 64), (2, 0, 64), (2, 1 << 20, 64), (2, 64, 1 << 20)):
        assert lib.moed_selftest_linear(*size, 0, 0, path) == md.MOED_ERR_SHAPE, size
    for types in ((2, 0), (0, -1)):
        assert lib.moed_selftest_linear(2, 64, 64, *types, path) == md.MOED_ERR_DTYPE
    assert lib.moed_selftest_linear(2, 64, 64, 0, 0, None) == md.MOED_ERR_NULL
    with pytest.raises(md.MoedError):
        md.moed_selftest_linear(0, 64, 64)
