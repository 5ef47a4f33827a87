"""Buffers that overlap are refused before anything is launched, by their ranges and not by their first bytes alone (no GPU
needed; the addresses are never read)."""
import ctypes

import pytest

from output_centric_expert_amd import moedecode as md
from test_abi import lib  # noqa: F401

P = ctypes.c_void_p
BF16, F32 = 0, 1
SIZE = {BF16: 2, F32: 4}


def place(sizes):
    """An address for each name, far from the others."""
    at, places = 1 << 20, {}
    for name, size in sizes.items():
        places[name] = at
        at += (size + (1 << 20)) & ~0xFFF
    return places


def shared(places, sizes, a, b):
    """Addresses of `a` that share a byte with `b`: the same one, the last 16 bytes of b, and a's end inside b."""
    end = places[b] + sizes[b] - 1
    return {places[b], end & ~0xF, (places[b] - sizes[a] + 16) & ~0xF}


class Linear:
    B, K, N = 64, 7168, 256

    def __init__(self, lib, x=F32, w=F32, bias=F32, residual=F32, out=F32):  # noqa: F811
        self.lib, self.types = lib, {"x": x, "w": w, "bias": bias, "residual": residual, "out": out}
        self.need = lib.moe_linear_workspace_bytes(self.B, self.K, self.N, x, w)
        B, K, N = self.B, self.K, self.N
        self.sizes = {"x": B * K * SIZE[x], "w": N * K * SIZE[w], "bias": N * SIZE[bias], "residual": B * N * SIZE[residual],
                      "out": B * N * SIZE[out], "workspace": max(self.need, 16)}
        self.places = place(self.sizes)

    def call(self, **places):
        p, t = {**self.places, **places}, self.types
        return self.lib.moe_linear(P(p["x"]), t["x"], P(p["w"]), t["w"], P(p["bias"]), t["bias"], 0, P(p["residual"]), t["residual"],
                                   P(p["out"]), t["out"], self.B, self.K, self.N, P(p["workspace"]), self.need, None)


@pytest.mark.parametrize("name", ["x", "w", "bias", "residual", "workspace"])
def test_linear_out_overlaps_nothing(lib, name):  # noqa: F811
    c = Linear(lib, out=BF16)
    assert c.need > 0
    for at in shared(c.places, c.sizes, "out", name):
        assert c.call(out=at) == md.MOED_ERR_SHAPE, (name, hex(at))


@pytest.mark.parametrize("residual,out", [(BF16, F32), (F32, BF16)])
def test_linear_in_place_needs_one_type(lib, residual, out):  # noqa: F811
    """Elements of other sizes lie elsewhere: a workgroup's outputs would be another's residual, still to be read."""
    c = Linear(lib, residual=residual, out=out)
    assert c.call(out=c.places["residual"]) == md.MOED_ERR_SHAPE


def test_linear_in_place_is_one_address(lib):  # noqa: F811
    c = Linear(lib)
    for off in (-16, 16, 1024):
        assert c.call(out=c.places["residual"] + off) == md.MOED_ERR_SHAPE


@pytest.mark.parametrize("name", ["x", "w", "bias", "residual", "out"])
def test_linear_workspace_overlaps_nothing(lib, name):  # noqa: F811
    c = Linear(lib)
    assert c.need > 0
    for at in shared(c.places, c.sizes, "workspace", name):
        assert c.call(workspace=at) == md.MOED_ERR_SHAPE, (name, hex(at))
