"""Host-side checks of the operators around the MoE block: bad arguments are refused before anything is launched
(no GPU needed; the addresses are never read)."""
import pytest

from output_centric_expert_amd import moedecode as md
from test_abi import A, MIS, lib  # noqa: F401


def linear(lib, x=A, xd=0, w=A, wd=0, b=A, bd=1, act=0, r=A, rd=0, out=A, od=0, B=2, K=64, N=64, ws=A, wsb=1 << 40):
    return lib.moe_linear(x, xd, w, wd, b, bd, act, r, rd, out, od, B, K, N, ws, wsb, None)


def test_linear_rejects(lib):  # noqa: F811
    assert linear(lib, B=0) == md.MOED_OK
    for kw in ({"B": -1}, {"B": 1 << 22}, {"K": 0}, {"N": 0}, {"K": 1 << 20}, {"N": 1 << 20}, {"K": 1 << 16, "N": 1 << 16},
               {"B": (1 << 22) - 1, "K": 1 << 19, "N": 8}, {"B": (1 << 22) - 1, "N": 1 << 19, "K": 8}):
        assert linear(lib, **kw) == md.MOED_ERR_SHAPE, kw
        assert lib.moe_linear_workspace_bytes(kw.get("B", 2), kw.get("K", 64), kw.get("N", 64), 0, 0) == 0
    for kw in ({"xd": 2}, {"wd": -1}, {"bd": 2}, {"rd": 2}, {"od": 2}, {"act": -1}, {"act": 7}):
        assert linear(lib, **kw) == md.MOED_ERR_DTYPE, kw
    for kw in ({"x": None}, {"w": None}, {"out": None}):
        assert linear(lib, **kw) == md.MOED_ERR_NULL, kw
    for name in ("x", "w", "r", "out"):
        assert linear(lib, **{name: MIS}) == md.MOED_ERR_ALIGN, name
    assert lib.moe_linear_workspace_bytes(2, 64, 64, 2, 0) == 0
    assert lib.moe_linear_workspace_bytes(2, 64, 64, 0, -1) == 0


@pytest.mark.parametrize("B,K,N", [(16, 7168, 256), (64, 7168, 256), (3, 65536, 1), (200, 20000, 40), (33, 4096, 4096)])
@pytest.mark.parametrize("xd,wd", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_linear_workspace(lib, B, K, N, xd, wd):  # noqa: F811
    need = lib.moe_linear_workspace_bytes(B, K, N, xd, wd)
    if need:
        assert linear(lib, B=B, K=K, N=N, xd=xd, wd=wd, ws=None) == md.MOED_ERR_NULL
        assert linear(lib, B=B, K=K, N=N, xd=xd, wd=wd, wsb=need - 1) == md.MOED_ERR_WORKSPACE
        assert linear(lib, B=B, K=K, N=N, xd=xd, wd=wd, ws=MIS, wsb=need) == md.MOED_ERR_ALIGN


def route(lib, lg=A, ld=1, bias=A, score=1, G=4, tg=2, gs=1, rn=1, B=2, E=64, k=8, ns=0, ids=A, w=A):
    return lib.moe_route_scored(lg, ld, bias, score, G, tg, gs, rn, B, E, k, ns, 1.0, ids, w, None)


def test_route_scored_rejects(lib):  # noqa: F811
    assert route(lib, B=0) == md.MOED_OK
    for kw in ({"B": -1}, {"B": 1 << 22}, {"E": 0}, {"E": 2052}, {"G": 0}, {"G": 3}, {"G": 65, "E": 130}, {"tg": 0}, {"tg": 5},
               {"k": 0}, {"k": 33}, {"k": 65, "E": 256}, {"ns": -1}, {"B": 1 << 21, "E": 1024}, {"B": 1 << 20, "ns": 1 << 11},
               {"ns": (1 << 31) - 1}):
        assert route(lib, **kw) == md.MOED_ERR_SHAPE, kw
    for kw in ({"ld": 2}, {"ld": -1}, {"score": 2}, {"score": -1}, {"gs": 2}, {"gs": -1}):
        assert route(lib, **kw) == md.MOED_ERR_DTYPE, kw
    for kw in ({"lg": None}, {"ids": None}, {"w": None}):
        assert route(lib, **kw) == md.MOED_ERR_NULL, kw


def post(lib, y=A, yd=0, R=4, pos=None, tw=None, k=2, pg=A, pgd=0, pe=1e-6, g=None, gd=0, gs=0, ga=0, r=A, rd=0, ro=A, gain=A,
         gaind=0, eps=1e-6, out=A, od=0, q=A, s=A, B=2, H=64):
    # out and residual_out are told apart by their addresses
    if out is A:
        out = A.value + 4096 if hasattr(A, "value") else A + 4096
    return lib.moe_post_norm(y, yd, R, pos, tw, k, pg, pgd, pe, g, gd, gs, ga, 1.0, r, rd, 1.0, ro, gain, gaind, eps, out, od,
                             q, s, B, H, None)


def test_post_norm_rejects(lib):  # noqa: F811
    assert post(lib, B=0) == md.MOED_OK
    for kw in ({"B": -1}, {"B": 1 << 22}, {"H": 0}, {"H": 32769}, {"H": 48}, {"eps": -1.0}, {"eps": float("nan")},
               {"pe": -1.0}, {"pe": float("nan")}, {"pos": A, "tw": A, "k": 0}, {"pos": A, "tw": A, "k": 65},
               {"pos": A, "tw": A, "R": -1}, {"pos": A, "tw": A, "R": 1 << 28}):
        assert post(lib, **kw) == md.MOED_ERR_SHAPE, kw
    for kw in ({"yd": 2}, {"rd": -1}, {"pgd": 7}, {"gaind": 2}, {"od": 2}, {"gs": 4}, {"gs": -1}, {"g": A, "gs": 1, "gd": 2},
               {"ga": 1}, {"ga": 2}, {"ga": 3}, {"ga": 4}, {"ga": 7}):
        assert post(lib, **kw) == md.MOED_ERR_DTYPE, kw
    for kw in ({"y": None}, {"r": None}, {"pos": A}, {"tw": A}, {"g": A}, {"gs": 1}, {"q": None}, {"s": None}, {"gain": None},
               {"gain": A, "out": None, "q": None, "s": None}, {"gain": None, "out": None, "q": None, "s": None, "ro": None},
               {"y": None, "pos": A, "tw": A, "R": 1}):
        assert post(lib, **kw) == md.MOED_ERR_NULL, kw
    for name in ("y", "pg", "r", "ro", "gain", "out", "q"):
        assert post(lib, **{name: MIS}) == md.MOED_ERR_ALIGN, name
    assert post(lib, g=MIS, gs=2) == md.MOED_ERR_ALIGN
    same = A.value + 4096 if hasattr(A, "value") else A + 4096
    assert post(lib, ro=same, out=A) == md.MOED_ERR_SHAPE
    # the experts' rows are not overwritten
    assert post(lib, pos=A, tw=A, ro=A) == md.MOED_ERR_SHAPE
    assert post(lib, pos=A, tw=A, ro=None, y=same) == md.MOED_ERR_SHAPE


def test_linear_outputs_overlap_nothing(lib):  # noqa: F811
    at = getattr(A, "value", A)
    need = lib.moe_linear_workspace_bytes(64, 7168, 256, 1, 1)
    assert need > 0
    for kw in ({"out": at}, {"x": at + 4096, "out": at + 4096, "ws": at + 8192}, {"w": at + 4096, "out": at + 4096, "ws": at + 8192},
               {"out": at + 4096, "ws": at + 4096}, {"out": at + 4096, "r": at + 8192, "ws": at + 8192}):
        assert linear(lib, B=64, K=7168, N=256, xd=1, wd=1, wsb=need, **kw) == md.MOED_ERR_SHAPE, kw
