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


class PostNorm:
    B, H, R, k = 6, 256, 20, 3

    def __init__(self, lib, rows=False, **types):  # noqa: F811
        self.lib, self.rows = lib, rows
        self.types = {"y": F32, "post_gain": F32, "gate": F32, "residual": F32, "gain": F32, "out": F32, **types}
        t = self.types
        t["residual_out"] = t["residual"]
        B, H = self.B, self.H
        self.sizes = {"y": (self.R if rows else B) * H * SIZE[t["y"]], "position": B * self.k * 4, "topk_w": B * self.k * 4,
                      "post_gain": H * SIZE[t["post_gain"]], "gate": B * H * SIZE[t["gate"]], "residual": B * H * SIZE[t["residual"]],
                      "gain": H * SIZE[t["gain"]], "residual_out": B * H * SIZE[t["residual"]], "out": B * H * SIZE[t["out"]],
                      "out_q": B * H, "out_s": B * H // 32}
        self.places = place(self.sizes)

    def call(self, gate_shape=3, **places):
        p, t = {**self.places, **places}, self.types
        pos, tw = (P(p["position"]), P(p["topk_w"])) if self.rows else (None, None)
        return self.lib.moe_post_norm(P(p["y"]), t["y"], self.R, pos, tw, self.k, P(p["post_gain"]), t["post_gain"], 1e-6, P(p["gate"]),
                                      t["gate"], gate_shape, 0, 1.0, P(p["residual"]), t["residual"], 1.0, P(p["residual_out"]),
                                      P(p["gain"]), t["gain"], 1e-6, P(p["out"]), t["out"], P(p["out_q"]), P(p["out_s"]), self.B, self.H, None)


POST_OUT = ("residual_out", "out", "out_q", "out_s")
POST_IN = ("y", "post_gain", "gate", "residual", "gain")


@pytest.mark.parametrize("out", POST_OUT)
@pytest.mark.parametrize("name", POST_IN + POST_OUT)
def test_post_norm_outputs_overlap_nothing(lib, out, name):  # noqa: F811
    """But y [B][H] and the residual at the address and of the type of out or residual_out."""
    if name == out:
        return
    c = PostNorm(lib)
    legal = {c.places[name]} if name in ("y", "residual") and out in ("out", "residual_out") else set()
    for at in shared(c.places, c.sizes, out, name) - legal:
        assert c.call(**{out: at}) == md.MOED_ERR_SHAPE, hex(at)


@pytest.mark.parametrize("out", POST_OUT)
@pytest.mark.parametrize("name", POST_IN + ("position", "topk_w"))
def test_post_norm_of_rows_outputs_overlap_nothing(lib, out, name):  # noqa: F811
    c = PostNorm(lib, rows=True)
    legal = {c.places[name]} if name == "residual" and out in ("out", "residual_out") else set()
    for at in shared(c.places, c.sizes, out, name) - legal:
        assert c.call(**{out: at}) == md.MOED_ERR_SHAPE, hex(at)


@pytest.mark.parametrize("y,residual,out", [(BF16, F32, F32), (F32, BF16, BF16), (F32, F32, BF16), (BF16, BF16, F32)])
def test_post_norm_in_place_needs_one_type(lib, y, residual, out):  # noqa: F811
    c = PostNorm(lib, y=y, residual=residual, out=out)
    for a, b in (("out", "y"), ("out", "residual"), ("residual_out", "y")):
        if c.types[a] != c.types[b]:
            assert c.call(**{a: c.places[b]}) == md.MOED_ERR_SHAPE, (a, b)


@pytest.mark.parametrize("shape,size", [(1, 6), (2, 256), (3, 6 * 256)])
def test_post_norm_outputs_overlap_no_gate(lib, shape, size):  # noqa: F811
    """A gate is as long as its shape says."""
    c = PostNorm(lib, gate=BF16)
    last = (c.places["gate"] + size * 2 - 1) & ~0xF
    for out in POST_OUT:
        assert c.call(gate_shape=shape, **{out: last}) == md.MOED_ERR_SHAPE, out


@pytest.mark.parametrize("logits", [BF16, F32])
@pytest.mark.parametrize("out,name", [("ids", "logits"), ("ids", "bias"), ("ids", "w"), ("w", "logits"), ("w", "bias")])
def test_route_scored_outputs_overlap_nothing(lib, logits, out, name):  # noqa: F811
    B, E, k, shared_slots = 100, 64, 8, 1
    slots = B * (k + shared_slots) * 4
    sizes = {"logits": B * E * SIZE[logits], "bias": E * 4, "ids": slots, "w": slots}
    places = place(sizes)
    for at in shared(places, sizes, out, name):
        p = {**places, out: at}
        assert lib.moe_route_scored(P(p["logits"]), logits, P(p["bias"]), 1, 1, 1, 0, 1, B, E, k, shared_slots, 1.0, P(p["ids"]),
                                    P(p["w"]), None) == md.MOED_ERR_SHAPE, hex(at)
