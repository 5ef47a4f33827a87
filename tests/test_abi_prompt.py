"""Host-side checks of the prompt-side entry points: bad arguments are refused before anything is launched
(no GPU needed; the addresses are never read)."""
import ctypes

import pytest

from output_centric_expert_amd import moedecode as md
from test_abi import A, MIS, lib  # noqa: F401

OK_BIG = 1 << 40


def norm(lib, x=A, xd=0, r=A, rd=0, g=A, gd=0, eps=1e-6, ro=A, out=A, od=0, q=A, s=A, B=2, H=64):
    return lib.moe_norm(x, xd, r, rd, g, gd, eps, ro, out, od, q, s, B, H, None)


def test_norm_rejects(lib):  # noqa: F811
    assert norm(lib, B=0) == md.MOED_OK
    for kw in ({"B": -1}, {"B": 1 << 22}, {"H": 0}, {"H": 32769}, {"H": 48}, {"eps": -1.0}, {"eps": float("nan")}):
        assert norm(lib, **kw) == md.MOED_ERR_SHAPE, kw
    for kw in ({"xd": 2}, {"rd": -1}, {"gd": 7}, {"od": 2}):
        assert norm(lib, **kw) == md.MOED_ERR_DTYPE, kw
    for kw in ({"x": None}, {"g": None}, {"s": None}, {"q": None}, {"out": None, "q": None, "s": None}, {"r": None}):
        assert norm(lib, **kw) == md.MOED_ERR_NULL, kw
    for name in ("x", "r", "g", "ro", "out", "q"):
        assert norm(lib, **{name: MIS}) == md.MOED_ERR_ALIGN, name


def group(lib, ids=A, B=2, k=2, E=8, order=A, pos=A, off=A, ws=None, wsb=0):
    return lib.moe_group(ids, B, k, E, order, pos, off, ws, wsb, None)


def test_group_rejects(lib):  # noqa: F811
    for kw in ({"B": -1}, {"k": 0}, {"k": 65}, {"E": 0}, {"E": 2049}, {"B": 1 << 22}, {"B": (1 << 22) - 1, "k": 64}):
        if kw == {"B": (1 << 22) - 1, "k": 64}:
            assert (kw["B"] * kw["k"]) < 1 << 28          # just inside: refused for its workspace instead
            assert group(lib, **kw) == md.MOED_ERR_NULL
        else:
            assert group(lib, **kw) == md.MOED_ERR_SHAPE, kw
    for name in ("ids", "order", "pos", "off"):
        assert group(lib, **{name: None}) == md.MOED_ERR_NULL, name
    assert lib.moe_group_workspace_bytes(1024, 8, 128) == 0
    need = lib.moe_group_workspace_bytes(16384, 8, 128)
    assert need > 0 and need % (128 * 4) == 0
    assert lib.moe_group_workspace_bytes(-1, 8, 128) == 0
    assert group(lib, B=16384, k=8, E=128, ws=A, wsb=need - 1) == md.MOED_ERR_WORKSPACE
    assert group(lib, B=16384, k=8, E=128, ws=ctypes.c_void_p(4097), wsb=need) == md.MOED_ERR_ALIGN


def gate_up(lib, a=A, a_s=None, rows=0, n_a=8, order=A, k=2, off=A, wq=A, ws=A, uq=A, us=A, wf=0, out=A, out_s=None,
            out_rows=0, R=16, E=8, K=512, N=64, wsp=None, wsb=0):
    return lib.moe_grouped_gate_up(a, a_s, rows, n_a, order, k, off, wq, ws, uq, us, wf, out, out_s, out_rows, R, E, K, N,
                                   wsp, wsb, None)


def matmul(lib, a=A, a_s=None, rows=0, n_a=8, order=A, k=2, off=A, wq=A, ws=A, wf=0, out=A, out_rows=0, R=16, E=8, K=512,
           N=64, wsp=None, wsb=0):
    return lib.moe_grouped_matmul(a, a_s, rows, n_a, order, k, off, wq, ws, wf, out, out_rows, R, E, K, N, wsp, wsb, None)


@pytest.mark.parametrize("call", [gate_up, matmul])
def test_products_reject(lib, call):  # noqa: F811
    assert call(lib, R=0) == md.MOED_OK
    for kw in ({"R": -1}, {"R": 1 << 28}, {"n_a": -1}, {"n_a": 0}, {"k": 0}, {"E": 0}, {"E": 2049}, {"K": 48}, {"N": 40},
               {"K": 0}, {"N": 1 << 20}, {"order": None}, {"K": 1 << 16, "N": 1 << 16}, {"n_a": 1 << 22}, {"R": (1 << 28) - 1, "N": 8192}):
        assert call(lib, **kw) == md.MOED_ERR_SHAPE, kw
    for kw in ({"rows": 1}, {"rows": 3}, {"wf": 2}, {"out_rows": 3}, {"out_rows": -1}):
        assert call(lib, **kw) == md.MOED_ERR_DTYPE, kw
    for kw in ({"a": None}, {"off": None}, {"wq": None}, {"ws": None}, {"out": None}, {"rows": 2}, {"a_s": A}):
        assert call(lib, **kw) == md.MOED_ERR_NULL, kw
    for name in ("a", "wq", "out"):
        assert call(lib, **{name: MIS}) == md.MOED_ERR_ALIGN, name
    odd = ctypes.c_void_p(4098)
    assert call(lib, ws=odd) == md.MOED_ERR_ALIGN
    assert call(lib, rows=2, a_s=odd) == md.MOED_ERR_ALIGN
    # K = 64: two scales a row, in rows of 16 in the workspace
    need = lib.moe_grouped_workspace_bytes(8, 64, 64, 8, 0, 2 if call is gate_up else 1)
    assert need == 8 * 64 * (2 if call is gate_up else 1) * 16
    assert call(lib, K=64) == md.MOED_ERR_NULL
    assert call(lib, K=64, wsp=A, wsb=need - 1) == md.MOED_ERR_WORKSPACE
    assert call(lib, K=64, wsp=MIS, wsb=need) == md.MOED_ERR_ALIGN


def test_products_reject_more(lib):  # noqa: F811
    assert lib.moe_grouped_workspace_bytes(8, 64, 32, 5, 2, 1) == (8 * 32 + 5) * 16
    for args in ((8, 512, 32, 5, 2, 1), (8, 768, 32, 5, 0, 2), (8, 48, 32, 5, 0, 2), (8, 64, 32, 5, 0, 3)):
        assert lib.moe_grouped_workspace_bytes(*args) == 0
    assert matmul(lib, out_rows=2) == md.MOED_ERR_DTYPE
    assert gate_up(lib, out_rows=2) == md.MOED_ERR_NULL                  # codes without scales
    assert gate_up(lib, out_s=A) == md.MOED_ERR_NULL                     # scales without codes
    assert gate_up(lib, uq=None) == md.MOED_ERR_NULL
    assert gate_up(lib, us=None) == md.MOED_ERR_NULL
    assert gate_up(lib, uq=MIS) == md.MOED_ERR_ALIGN


def combine(lib, y=A, yd=0, R=16, pos=A, w=A, out=A, od=0, B=2, k=2, H=64):
    return lib.moe_combine(y, yd, R, pos, w, out, od, B, k, H, None)


def test_combine_rejects(lib):  # noqa: F811
    assert combine(lib, B=0) == md.MOED_OK
    for kw in ({"B": -1}, {"B": 1 << 22}, {"k": 0}, {"k": 65}, {"H": 0}, {"H": 1 << 20}, {"R": -1}, {"R": 1 << 28}):
        assert combine(lib, **kw) == md.MOED_ERR_SHAPE, kw
    for kw in ({"yd": 2}, {"od": 2}):
        assert combine(lib, **kw) == md.MOED_ERR_DTYPE, kw
    for name in ("y", "pos", "w", "out"):
        assert combine(lib, **{name: None}) == md.MOED_ERR_NULL, name
    for name in ("y", "out"):
        assert combine(lib, **{name: MIS}) == md.MOED_ERR_ALIGN, name


def prefill(lib, x=A, x_s=None, rows=0, ids=A, w=A, q=A, s=A, wf=0, out=A, od=0, B=2, E=8, k=2, H=64, I=32, ws=A,
            wsb=OK_BIG):
    return lib.moe_prefill(x, x_s, rows, ids, w, q, s, q, s, q, s, wf, out, od, B, E, k, H, I, ws, wsb, None)


def test_prefill_rejects(lib):  # noqa: F811
    assert prefill(lib, B=0) == md.MOED_OK
    for kw in ({"B": -1}, {"B": 1 << 22}, {"E": 0}, {"E": 2049}, {"k": 9}, {"k": 0}, {"H": 40}, {"I": 0}, {"I": 33}):
        assert prefill(lib, **kw) == md.MOED_ERR_SHAPE, kw
    for kw in ({"rows": 1}, {"wf": 2}, {"od": 2}):
        assert prefill(lib, **kw) == md.MOED_ERR_DTYPE, kw
    for kw in ({"x": None}, {"ids": None}, {"w": None}, {"q": None}, {"s": None}, {"out": None}, {"ws": None},
               {"x_s": A}, {"rows": 2}):
        assert prefill(lib, **kw) == md.MOED_ERR_NULL, kw
    for name in ("x", "q", "out", "ws"):
        assert prefill(lib, **{name: MIS}) == md.MOED_ERR_ALIGN, name
    need = lib.moe_prefill_workspace_bytes(2, 8, 2, 64, 32, 0, 0)
    assert prefill(lib, wsb=need - 1) == md.MOED_ERR_WORKSPACE
    # order, position, offsets, the gate and up scales in rows of 16, bfloat16 intermediate, bfloat16 rows, each
    # rounded up to 256 bytes
    assert need == 256 + 256 + 256 + 2 * 8 * 32 * 16 + 256 + 512
    # float32 out: MXFP8 intermediate and its scales; the tokens' scales beside the matrices'
    assert lib.moe_prefill_workspace_bytes(2, 8, 2, 64, 32, 2, 1) == 256 * 3 + (2 * 8 * 32 * 16 + 256) + 256 + 256 + 1024
    assert lib.moe_prefill_workspace_bytes(2, 8, 2, 512, 640, 0, 0) == 256 * 3 + 4 * 640 * 2 + 4 * 512 * 2
    assert lib.moe_prefill_workspace_bytes(0, 8, 2, 64, 32, 0, 0) == 0
    assert lib.moe_prefill_workspace_bytes(2, 8, 2, 64, 33, 0, 0) == 0
