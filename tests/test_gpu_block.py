"""GPU tests of the operators around the MoE block (moe_linear, moe_route_scored, moe_post_norm) against plain float64
computations.

Products are tested two ways: with whole numbers, for which every float32 sum is exact and the result has to be equal
bit for bit, whatever tile, split or order a size takes, and with normal values against the bound of a float32 sum: n
terms in any order are off by at most n * 2^-24 * sum |terms| to first order; the matrix instructions may truncate where
an addition would round, so 2^-23 per term is allowed, and 2^-23 of each term for the parts that the product of two
float32 values leaves out. A store to bfloat16 is off by at most 2^-8 of the value (half a step). What is chosen by the
router has to be equal; its weights are one rounding (2^-24) of numbers computed in 64 bits."""
import math

import numpy as np
import pytest
import torch

from output_centric_expert_amd import moedecode as md

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
ACTS = (None, "silu", "gelu", "gelu_tanh", "relu", "sigmoid", "tanh")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    md.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


# ---------------------------------------------------------------------------- linear

def act64(v, act):
    F = torch.nn.functional
    return {None: lambda t: t, "silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda t: F.gelu(t, approximate="tanh"),
            "relu": torch.relu, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[act](v)


def check_linear(x, w, bias, act, residual, out):
    v = x.double() @ w.double().T
    tol = (x.shape[1] + 8) * 2 * U * (x.double().abs() @ w.double().abs().T)
    if bias is not None:
        v = v + bias.double()
        tol = tol + U * v.abs()
    # no activation is steeper than 1.13; its own float32 steps (exp and erfc to a few units in the last place)
    tol = 1.13 * tol + 48 * U * v.abs().clamp(min=1) * (act is not None)
    v = act64(v, act)
    if residual is not None:
        v = v + residual.double()
        tol = tol + U * v.abs()
    tol = tol + STEP[out.dtype] * v.abs() + 1e-37
    off = (out.double() - v).abs()
    assert (off <= tol).all(), float((off / tol).max())


SIZES = [(1, 1, 1), (1, 2048, 128), (1, 7168, 256), (2, 33, 5), (3, 1111, 777), (4, 8, 4096), (5, 4096, 1), (7, 100, 300),
         (8, 2048, 512), (9, 512, 16), (16, 7168, 256), (17, 63, 65), (31, 2049, 130), (32, 4096, 1024), (33, 64, 33),
         (64, 7168, 256), (65, 200, 257), (127, 1000, 96), (128, 128, 128), (200, 20000, 40), (256, 256, 512), (300, 1, 300),
         (1000, 1111, 777), (513, 4104, 520), (2048, 96, 8), (2500, 7, 3), (1024, 1024, 1024), (4096, 520, 264), (4100, 264, 4100), (4100, 77, 4099),
         # tiles with K even and odd, with k whole and split, steps that end behind K and that do not (not every way of
         # every tile: linear_paths.py has the rest)
         (4090, 712, 4093), (4090, 711, 4093), (4096, 256, 4096), (3161, 37, 2629), (4272, 34, 899), (3692, 33, 1028),
         (2052, 2877, 900), (3422, 34, 546), (647, 33, 2967), (4107, 2212, 35), (3291, 2871, 34), (34, 34, 3285), (33, 33, 3425),
         (36, 998, 3244), (3225, 1189, 33), (2369, 33, 1717), (133, 2816, 3586), (3943, 2765, 130), (3491, 850, 33),
         (36, 887, 3461), (2299, 35, 1812), (2765, 1296, 641), (808, 1319, 2466), (3427, 884, 33), (34, 971, 3354),
         (4340, 2106, 71), (259, 37, 3333), (35, 604, 3665), (33, 613, 3401), (3271, 40, 37), (34, 1292, 3557), (36, 1325, 3674),
         (18, 1492, 20), (18, 1561, 19), (19, 1724, 18), (19, 1963, 18), (20, 890, 18), (21, 789, 18),
         # the same of the kernel of few rows
         (5, 9001, 40), (2000, 9001, 7), (400, 9004, 16), (40, 5001, 24), (24, 5003, 100), (6, 9002, 40), (3000, 200, 20), (3001, 201, 30)]


@pytest.mark.parametrize("B,K,N", SIZES)
@pytest.mark.parametrize("x_type,w_type", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_linear(B, K, N, x_type, w_type):
    g = gen(B * 31 + K * 7 + N)
    x, w = randn(g, B, K).to(TYPES[x_type]), (randn(g, N, K) / math.sqrt(K)).to(TYPES[w_type])
    out = md.moe_linear(x, w, out_dtype=torch.float32)
    check_linear(x, w, None, None, None, out)
    bias, residual = randn(g, N), randn(g, B, N)
    act = ACTS[(B + N) % len(ACTS)]
    for bt, rt, ot in (("f32", "bf16", "bf16"), ("bf16", "f32", "f32")):
        b, r = bias.to(TYPES[bt]), residual.to(TYPES[rt])
        check_linear(x, w, b, act, r, md.moe_linear(x, w, bias=b, activation=act, residual=r, out_dtype=TYPES[ot]))


@pytest.mark.parametrize("B,K,N", SIZES)
@pytest.mark.parametrize("x_type,w_type", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_linear_whole_numbers(B, K, N, x_type, w_type):
    """Sums of whole numbers below 2^24: exact. Float32 operands hold numbers that no bfloat16 does."""
    g = gen(B + K + N)
    if K > 5000:
        K = K // 4 + 1
    big = 1000 if x_type != w_type or x_type == "f32" else 3
    x = torch.randint(-(big if x_type == "f32" else 3), (big if x_type == "f32" else 3) + 1, (B, K), generator=g, device="cuda")
    top = big if w_type == "f32" and x_type != "f32" else 3
    w = torch.randint(-top, top + 1, (N, K), generator=g, device="cuda")
    ref = (x.double() @ w.double().T).float()
    bias = torch.randint(-9, 10, (N,), generator=g, device="cuda")
    res = torch.randint(-99, 100, (B, N), generator=g, device="cuda")
    xv, wv = x.to(TYPES[x_type]), w.to(TYPES[w_type])
    assert torch.equal(md.moe_linear(xv, wv, out_dtype=torch.float32), ref)
    out = md.moe_linear(xv, wv, bias=bias.float(), activation="relu", residual=res.bfloat16(), out_dtype=torch.float32)
    assert torch.equal(out, torch.relu(ref + bias) + res)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("B", [1, 40])
def test_linear_activations(B, act):
    """Arguments from -100 to 100 through every activation (the product is with one)."""
    v = torch.linspace(-100, 100, 2001, device="cuda")[:, None]
    out = md.moe_linear(torch.ones(B, 1, device="cuda"), v, activation=act, out_dtype=torch.float32)
    ref = act64(v.double().T, act).expand(B, -1)
    tol = 48 * U * v.double().T.abs().clamp(min=1) if act else 0 * ref
    assert ((out.double() - ref).abs() <= tol).all()
    # away from zero these lose no relative precision to cancellation
    if act in ("silu", "gelu_tanh", "sigmoid"):
        near = (v.T.abs() < 5).expand(B, -1)
        assert ((out.double() - ref).abs()[near] <= 2.0 ** -17 * ref.abs()[near]).all()


@pytest.mark.parametrize("B", [1, 6, 40, 300])
@pytest.mark.parametrize("w_type", ["bf16", "f32"])
def test_linear_in_place_and_neighbours(B, w_type):
    """residual = out; rows of the buffer in front of and behind the result stay as they were."""
    g = gen(B)
    x, w = randn(g, B, 200).bfloat16(), randn(g, 72, 200).to(TYPES[w_type])
    buf = randn(g, B + 16, 72)
    before = buf.clone()
    out = buf[8:B + 8]
    ref = md.moe_linear(x, w, residual=out.clone(), out_dtype=torch.float32)
    assert md.moe_linear(x, w, residual=out, out=out) is out
    assert torch.equal(bits(out), bits(ref))
    assert torch.equal(buf[:8], before[:8]) and torch.equal(buf[B + 8:], before[B + 8:])


@pytest.mark.parametrize("B,K,N", [(1, 64, 77), (40, 9000, 77), (300, 64, 500), (2052, 2877, 904)])
@pytest.mark.parametrize("bias_type", ["bf16", "f32"])
def test_linear_bias_at_any_element(B, K, N, bias_type):
    g = gen(B + N)
    x, w, b = randn(g, B, K), randn(g, N, K) / math.sqrt(K), randn(g, N + 9).to(TYPES[bias_type])
    for at in (1, 3, 8):
        part = b[at:at + N]
        assert torch.equal(bits(md.moe_linear(x, w, bias=part, out_dtype=torch.float32)),
                           bits(md.moe_linear(x, w, bias=part.clone(), out_dtype=torch.float32)))


@pytest.mark.parametrize("B", [1, 8, 40, 300])
@pytest.mark.parametrize("x_type,w_type", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_linear_special_values(B, x_type, w_type):
    """A NaN or an infinity enters the outputs of its row of x, or of w, and no others."""
    g = gen(B + 3)
    for K in (64, 77, 512):
        x, w = randn(g, B, K).to(TYPES[x_type]), randn(g, 40, K).to(TYPES[w_type])
        ref = md.moe_linear(x, w, out_dtype=torch.float32)
        for bad in (float("nan"), float("inf"), -float("inf")):
            x2, w2 = x.clone(), w.clone()
            x2[B // 2, K - 1] = bad
            out = md.moe_linear(x2, w, out_dtype=torch.float32)
            assert not out[B // 2].isfinite().any()
            keep = torch.arange(B, device="cuda") != B // 2
            assert torch.equal(out[keep], ref[keep])
            w2[39, 0] = bad
            out = md.moe_linear(x, w2, out_dtype=torch.float32)
            assert not out[:, 39].isfinite().any() and torch.equal(out[:, :39], ref[:, :39])


@pytest.mark.parametrize("power", [-100, -60, 60, 100])
@pytest.mark.parametrize("B", [2, 64])
def test_linear_far_values(B, power):
    """float32 operands far from one: x times 2^power, w times 2^-power is the same product."""
    g = gen(77)
    x, w = randn(g, B, 256), randn(g, 48, 256)
    a = md.moe_linear(x, w, out_dtype=torch.float32)
    b = md.moe_linear(torch.ldexp(x, torch.tensor(power, device="cuda")), torch.ldexp(w, torch.tensor(-power, device="cuda")),
                      out_dtype=torch.float32)
    # at 2^-100 the lowest part of a value may be a subnormal bfloat16, whose steps are 2^-133: 2^-33 of the value's unit
    assert ((a - b).abs().double() <= 256 * 2 * U * (x.double().abs() @ w.double().abs().T)).all()


@pytest.mark.parametrize("B,K,N", [(1, 77, 5), (5, 77, 40), (40, 1111, 40), (40, 65, 7), (300, 77, 500), (300, 1028, 500),
                                   (300, 1029, 500), (2000, 33, 700), (4090, 201, 4090)])
@pytest.mark.parametrize("x_type,w_type", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_linear_reads_and_writes_nothing_behind(B, K, N, x_type, w_type):
    """NaN in front of and behind x, w, bias and residual changes nothing; what lies around out stays."""
    g = gen(B + K + N)

    def inside(t):
        buf = torch.full((t.numel() + 1024,), float("nan"), device="cuda", dtype=t.dtype)
        buf[512:512 + t.numel()] = t.reshape(-1)
        return buf[512:512 + t.numel()].view(t.shape)

    x, w, b, r = randn(g, B, K).to(TYPES[x_type]), randn(g, N, K).to(TYPES[w_type]), randn(g, N), randn(g, B, N)
    for dt in TYPES.values():
        ref = md.moe_linear(x, w, bias=b, residual=r.to(dt), out_dtype=dt)
        buf = torch.full((B * N + 1024,), 7.0, device="cuda", dtype=dt)
        out = buf[512:512 + B * N].view(B, N)
        md.moe_linear(inside(x), inside(w), bias=inside(b), residual=inside(r.to(dt)), out=out)
        assert torch.equal(bits(out), bits(ref)) and (buf[:512] == 7).all() and (buf[512 + B * N:] == 7).all()


@pytest.mark.parametrize("B,K,N,x_type,w_type", [(300000, 8192, 16, "bf16", "bf16"), (300000, 8192, 40, "bf16", "bf16"),
                                                 (300000, 8190, 300, "bf16", "f32"), (150000, 8191, 40, "f32", "bf16"),
                                                 (40, 4096, 600000, "bf16", "bf16"), (3, 4097, 600000, "bf16", "bf16"),
                                                 (1, 4097, 600000, "bf16", "f32"), (9000, 64, 300000, "bf16", "bf16"),
                                                 (5, (1 << 20) - 1, 40, "bf16", "f32"), (300, (1 << 20) - 3, 300, "bf16", "bf16")])
def test_linear_past_32_bits(B, K, N, x_type, w_type):
    """Operands and outputs past 4 GiB, rows of a million values: outputs at the ends and at random places."""
    g = gen(11)
    x = torch.empty(B, K, device="cuda", dtype=TYPES[x_type])
    w = torch.empty(N, K, device="cuda", dtype=TYPES[w_type])
    for t in (x, w):
        for part in t.split(1 << 14):
            part.copy_(torch.randint(-2, 3, part.shape, generator=g, device="cuda"))
    out = md.moe_linear(x, w, out_dtype=torch.bfloat16 if B * N > 1 << 30 else torch.float32)
    rows = torch.cat([torch.arange(min(B, 3)), torch.arange(max(0, B - 3), B), torch.randint(0, B, (40,))]).unique().cuda()
    cols = torch.cat([torch.arange(min(N, 3)), torch.arange(max(0, N - 3), N), torch.randint(0, N, (200,))]).unique().cuda()
    ref = x[rows].double() @ w[cols].double().T               # whole numbers below 2^24: exact
    assert torch.equal(out[rows][:, cols], ref.to(out.dtype))


def test_linear_repeats():
    """The same call gives the same bits."""
    g = gen(5)
    for B, K, N in ((64, 7168, 256), (32, 4096, 1024), (300, 1111, 100)):
        x, w = randn(g, B, K).bfloat16(), randn(g, N, K)
        a = md.moe_linear(x, w, out_dtype=torch.float32)
        for _ in range(3):
            assert torch.equal(bits(a), bits(md.moe_linear(x, w, out_dtype=torch.float32)))


def test_linear_empty_and_refusals():
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(8, 64, device="cuda")
    assert md.moe_linear(x, w).shape == (0, 8)
    x = torch.ones(4, 64, device="cuda")
    for kw, err in (({"activation": "swish"}, ValueError), ({"out_dtype": torch.float16}, TypeError),
                    ({"bias": torch.ones(9, device="cuda")}, ValueError), ({"residual": torch.ones(4, 9, device="cuda")}, ValueError),
                    ({"out": torch.ones(4, 8)}, ValueError), ({"residual": torch.ones(8, 4, device="cuda").T}, ValueError)):
        with pytest.raises(err):
            md.moe_linear(x, w, **kw)
    with pytest.raises(TypeError):
        md.moe_linear(x.half(), w)
    with pytest.raises(ValueError):
        md.moe_linear(x.T, torch.ones(8, 4, device="cuda"))
    with pytest.raises(ValueError):
        md.moe_linear(x, w[:, :63])
    with pytest.raises(md.MoedError):                         # an address between 16-byte borders
        md.moe_linear(torch.ones(257, device="cuda")[1:].view(4, 64), w)
    need = md.moe_linear_workspace_bytes(64, 7168, 256, torch.bfloat16, torch.float32)
    if need:
        with pytest.raises(md.MoedError):
            md.moe_linear(torch.ones(64, 7168, device="cuda").bfloat16(), torch.ones(256, 7168, device="cuda"),
                          workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------------------- route

def route_ref(logits, k, score, bias, G, take, group_score, renorm, n_shared, scale):
    """The definition in numpy: float64 scores rounded to float32, choices in float32."""
    B, E = logits.shape
    x = logits.astype(np.float64)
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = np.where(np.isnan(x), -np.inf, x).max(1, keepdims=True)
            e = np.where(np.isnan(x), 0.0, np.where(x == m, 1.0, np.exp(x - m)))
            s = (e / e.sum(1, keepdims=True)).astype(np.float32)
        else:
            s = (1 / (1 + np.exp(-x))).astype(np.float32)
        c = s if bias is None else s + bias
    c = np.where(np.isnan(x) | np.isnan(c), -np.inf, c).astype(np.float32)
    if take < G:
        grouped = np.sort(c.reshape(B, G, E // G), axis=2)[:, :, ::-1]
        value = grouped[:, :, 0].copy()
        if group_score == "top2" and E > G:
            two = grouped[:, :, 1] > -np.inf
            value[two] = (grouped[:, :, 0] + np.where(two, grouped[:, :, 1], 0)).astype(np.float32)[two]
        order = np.argsort(-value, axis=1, kind="stable")
        closed = np.ones((B, G), bool)
        for b in range(B):
            for g in order[b, :take]:
                closed[b, g] = value[b, g] == -np.inf
        c = np.where(np.repeat(closed, E // G, axis=1), -np.inf, c)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    ok = np.take_along_axis(c, ids, 1) > -np.inf
    w = np.take_along_axis(s, ids, 1).astype(np.float64)
    if renorm:
        w = w / (np.where(ok, w, 0).sum(1, keepdims=True) + 1e-20)
    w = np.where(ok, w * np.float32(scale).astype(np.float64), np.nan)
    ids = np.where(ok, ids, -1)
    shared = np.broadcast_to(np.arange(E, E + n_shared), (B, n_shared))
    return np.concatenate([ids, shared], 1), np.concatenate([w, np.ones((B, n_shared))], 1)


def check_route(logits, k, score="sigmoid", bias=None, G=1, take=1, group_score="top2", renorm=True, n_shared=0, scale=1.0):
    ids, w = md.moe_route_scored(logits, k, score=score, bias=bias, n_group=G, topk_group=take, group_score=group_score,
                                 renormalize=renorm, n_shared=n_shared, routed_scale=scale)
    rid, rw = route_ref(logits.float().cpu().numpy(), k, score, None if bias is None else bias.cpu().numpy(), G, take,
                        group_score, renorm, n_shared, scale)
    assert np.array_equal(ids.cpu().numpy(), rid)
    w = w.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(w), np.isnan(rw))
    f = ~np.isnan(rw)
    # one rounding, and 2^-149 where a weight is subnormal
    assert (np.abs(w[f] - rw[f]) <= 1.01 * U * np.abs(rw[f]) + 2.0 ** -149).all()
    return ids, w


ROUTES = [(1, 128, 8, 1, 1), (64, 256, 8, 8, 4), (5, 8, 2, 4, 2), (3, 67, 5, 1, 1), (33, 160, 6, 8, 3), (2, 2048, 16, 16, 5),
          (4, 130, 64, 2, 2), (7, 1, 1, 1, 1), (9, 64, 64, 64, 64), (6, 512, 8, 64, 7), (257, 96, 4, 3, 1), (1000, 60, 7, 5, 2),
          (3000, 256, 8, 8, 4), (4100, 128, 8, 1, 1), (2049, 12, 3, 4, 2), (2100, 330, 5, 10, 9), (5000, 64, 1, 16, 1),
          (3, 2048, 64, 64, 3), (1030, 1024, 10, 32, 31)]


@pytest.mark.parametrize("B,E,k,G,take", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_scored(B, E, k, G, take, score, group_score):
    g = gen(B + E * 3 + k)
    logits, bias = 2 * randn(g, B, E), 0.1 * randn(g, E)
    check_route(logits, k, score, bias, G, take, group_score, True, 1, 2.5)
    check_route(logits, k, score, None, G, take, group_score, False, 0, 1.0)
    # bfloat16 logits: many are equal
    check_route(logits.bfloat16(), k, score, None, G, take, group_score, True, 2, 1.0)
    check_route(logits.bfloat16(), k, score, bias, G, take, group_score, False)


def test_route_scored_ties():
    """Equal choices and equal groups go to the lower index, also where few values occur at all."""
    g = gen(3)
    for E, G, take, k in ((64, 8, 3, 8), (256, 8, 4, 8), (100, 1, 1, 7), (512, 32, 9, 33)):
        logits = torch.randint(-1, 2, (500, E), generator=g, device="cuda").float()
        bias = torch.randint(-1, 2, (E,), generator=g, device="cuda").float() / 4
        for score in ("softmax", "sigmoid"):
            for b in (None, bias):
                check_route(logits, k, score, b, G, take)
        ids, _ = check_route(torch.zeros(70, E, device="cuda"), k, "softmax", None, G, take)
        assert torch.equal(ids.cpu(), torch.arange(k, dtype=torch.int32).expand(70, k))
    check_route(torch.tensor([[0.0, -0.0, 0.0, -0.0]], device="cuda"), 3, bias=torch.tensor([-0.5, -0.5, -0.5, -0.5], device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B", [12, 3000])
def test_route_scored_special_values(score, B):
    """NaN, infinite and far logits; masked experts, masked groups, masked rows; biases that mask."""
    g = gen(8)
    inf, nan = float("inf"), float("nan")
    for E, G, take, k in ((64, 8, 3, 8), (256, 8, 4, 8), (30, 5, 2, 6), (20, 20, 4, 2), (500, 10, 3, 9)):
        x = 2 * randn(g, B, E)
        x[0] = nan                                            # nothing can be chosen
        x[1] = -inf
        x[2] = inf
        x[3, ::2] = nan
        x[4, : E - 3] = nan                                   # fewer than k are left
        x[5, 1] = inf
        x[6, ::3] = -inf
        x[7] = torch.finfo(torch.float32).min
        x[8] *= 1e4                                           # scores of 0 and 1, subnormal ones
        x[9] = -95 + 3 * x[9]
        x[10, : E // G] = nan                                 # a group without any
        x[11, 1: E // G] = nan                                # a group with one
        bias = 0.1 * randn(g, E)
        bias[3], bias[4], bias[5] = -inf, nan, inf
        bias[E // G * 2: E // G * 3] = -inf
        for b in (None, bias):
            for gs in ("max", "top2"):
                for renorm in (False, True):
                    check_route(x, k, score, b, G, take, gs, renorm, 1, 0.5)
                    check_route(x, k, score, b, G, G, gs, renorm)


def test_route_scored_many_tokens():
    """As many tokens as the limit lets through, logits past 4 GiB."""
    B, E = (1 << 22) - 1, 511
    logits = torch.empty(B, E, device="cuda")
    for part in logits.split(1 << 18):
        part.normal_(generator=gen(part.data_ptr() % 1000))
    for k, G, take in ((8, 1, 1), (2, 7, 3)):
        ids, w = md.moe_route_scored(logits, k, n_group=G, topk_group=take)
        for rows in (slice(0, 40), slice(B - 40, B), slice(2103000, 2103040)):
            rid, rw = route_ref(logits[rows].cpu().numpy(), k, "sigmoid", None, G, take, "top2", True, 0, 1.0)
            assert np.array_equal(ids[rows].cpu().numpy(), rid) and np.allclose(w[rows].cpu().numpy(), rw, rtol=2 * U, atol=0)
    del logits
    logits = randn(gen(4), (1 << 22) - 1, 200)                # the kernel for many tokens, an odd count of them
    ids, w = md.moe_route_scored(logits, 8, n_group=8, topk_group=4)
    for rows in (slice(0, 40), slice((1 << 22) - 41, (1 << 22) - 1)):
        rid, rw = route_ref(logits[rows].cpu().numpy(), 8, "sigmoid", None, 8, 4, "top2", True, 0, 1.0)
        assert np.array_equal(ids[rows].cpu().numpy(), rid) and np.allclose(w[rows].cpu().numpy(), rw, rtol=2 * U, atol=0)


def test_route_scored_is_route():
    """Softmax without bias and groups, renormalised: moe_route's experts and weights."""
    logits = randn(gen(9), 500, 128) * 3
    ids, w = md.moe_route_scored(logits, 8, score="softmax", n_shared=1, routed_scale=1.5)
    ids2, w2 = md.moe_route(logits, 8, n_shared=1, routed_scale=1.5)
    assert torch.equal(ids, ids2)
    assert ((w - w2).abs() <= 1e-5 * w2).all()


def test_route_scored_empty_buffers_and_refusals():
    assert md.moe_route_scored(torch.empty(0, 64, device="cuda"), 8)[0].shape == (0, 8)
    logits = randn(gen(1), 5, 64)
    ids, w = torch.full((7, 9), 99, dtype=torch.int32, device="cuda"), torch.full((7, 9), 99.0, device="cuda")
    a, b = md.moe_route_scored(logits, 8, n_shared=1, ids=ids[1:6], w=w[1:6])
    assert a.data_ptr() == ids[1].data_ptr() and (ids[[0, 6]] == 99).all() and (w[[0, 6]] == 99).all() and (a != 99).all()
    for kw, err in (({"k": 65}, md.MoedError), ({"k": 0}, md.MoedError), ({"n_group": 3}, md.MoedError), ({"topk_group": 2}, md.MoedError),
                    ({"score": "tanh"}, ValueError), ({"group_score": "sum"}, ValueError), ({"n_shared": -1}, ValueError),
                    ({"bias": torch.ones(64, device="cuda").bfloat16()}, TypeError), ({"bias": torch.ones(65, device="cuda")}, ValueError),
                    ({"n_group": 8, "topk_group": 1, "k": 9}, md.MoedError)):
        with pytest.raises(err):
            md.moe_route_scored(logits, **{"k": 8, **kw})
    with pytest.raises(TypeError):
        md.moe_route_scored(logits.double(), 8)


# ---------------------------------------------------------------------------- post norm

def quantize(y):
    """Float32 [..., K] -> codes and scales by the rule of moe_norm, from the bits."""
    b = y.unflatten(-1, (-1, 32))
    field = (b.abs().view(torch.int32).amax(-1)) >> 23
    scale = torch.where(field == 255, torch.full_like(field, 255), (field - 8).clamp(min=0))
    t = torch.ldexp(b.double(), (127 - scale)[..., None].double()).clamp(-448, 448)
    q = t.float().to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.where((scale == 255)[..., None], torch.full_like(q, 0x7F), q)
    return q.flatten(-2), scale.to(torch.uint8)


def post_ref(y, residual, post_gain, post_eps, gate, gate_act, scale, residual_scale, gain, eps, position, topk_w):
    """(out, s) in float64 and the bounds of what float32 makes of them."""
    H = residual.shape[1]
    if position is not None:
        rows = y.double()[position.long()] * topk_w.double()[..., None]
        y, ey = rows.sum(1), (position.shape[1] + 1) * U * rows.abs().sum(1)
    else:
        y = y.double()
        ey = 0 * y
    if post_gain is not None:
        root = torch.sqrt((y * y).mean(1, keepdim=True) + post_eps)
        # the row's sum of squares (its error halved by the root), root, products; the error of y in itself and in the root
        e_root = (H / 2 + 10) * U + torch.sqrt((ey * ey).mean(1, keepdim=True)) / root
        t = y / root * post_gain.double()
        et = ey / root * post_gain.double().abs() + e_root * t.abs()
    else:
        t, et = y, ey
    f = torch.full_like(t, float(np.float32(scale)))
    if gate is not None:
        a = gate.double()
        f = f * act64(a, gate_act)
    r = float(np.float32(residual_scale)) * residual.double()
    s = r + f * t
    es = f.abs() * et + 24 * U * (f * t).abs() + U * r.abs() + U * s.abs()
    if gain is None:
        return None, s, None, es
    root = torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    out = s / root * gain.double()
    e_root = (H / 2 + 10) * U + torch.sqrt((es * es).mean(1, keepdim=True)) / root
    return out, s, es / root * gain.double().abs() + e_root * out.abs(), es


def check_post(y, residual, out_type=torch.float32, quant=False, **kw):
    full = {"post_gain": None, "post_eps": 1e-6, "gate": None, "gate_act": None, "scale": 1.0, "residual_scale": 1.0, "gain": None,
            "eps": 1e-6, "position": None, "topk_w": None, **kw}
    out, res, q, s = md.moe_post_norm(y, residual, out_dtype=out_type, quantize=quant, **kw)
    ref, sref, eout, es = post_ref(y, residual, **full)
    off = (res.double() - sref).abs()
    tol = 1.001 * es + STEP[res.dtype] * sref.abs() + 1e-37
    assert res.dtype == residual.dtype and (off <= tol).all(), float((off / tol).max())
    if full["gain"] is None:
        assert out is None and q is None and s is None
        return res
    off = (out.double() - ref).abs()
    tol = 1.001 * eout + STEP[out.dtype] * ref.abs() + 1e-37
    assert (off <= tol).all(), float((off / tol).max())
    if quant:
        rq, rs = quantize(out if out_type == torch.float32 else
                          md.moe_post_norm(y, residual, out_dtype=torch.float32, **kw)[0])
        assert torch.equal(s, rs) and torch.equal(q, rq)
    return out


def a_gate(g, shape, B, H, dtype):
    return None if shape is None else randn(g, *{"token": (B, 1), "channel": (H,), "full": (B, H)}[shape]).to(dtype)


@pytest.mark.parametrize("B,H", [(1, 1), (1, 2048), (3, 31), (5, 256), (2, 1111), (7, 4096), (2, 4104), (3, 7168), (2, 8192),
                                 (1, 8200), (2, 16416), (1, 32768), (1, 32767), (2500, 96), (2049, 2048), (3000, 250)])
@pytest.mark.parametrize("y_type,r_type", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_post_norm(B, H, y_type, r_type):
    g = gen(B * 131 + H)
    y, r = 2 * randn(g, B, H).to(TYPES[y_type]), 3 * randn(g, B, H).to(TYPES[r_type])
    gains = [(1 + 0.3 * randn(g, H)).to(t) for t in (torch.bfloat16, torch.float32)]
    quant = H % 32 == 0
    check_post(y, r, quant=quant, post_gain=gains[0], gain=gains[1], scale=0.7, residual_scale=0.9)
    check_post(y, r, out_type=torch.bfloat16, quant=quant, gain=gains[0], eps=1e-3)
    check_post(y, r, post_gain=gains[1], post_eps=1e-2)
    for shape, act, t in (("token", "sigmoid", torch.bfloat16), ("channel", "tanh", torch.float32), ("full", None, torch.bfloat16),
                          ("full", "sigmoid", torch.float32), ("token", None, torch.float32), ("channel", None, torch.bfloat16)):
        check_post(y, r, quant=quant, post_gain=gains[0], gain=gains[0], gate=a_gate(g, shape, B, H, t), gate_act=act, scale=1.3)


@pytest.mark.parametrize("B,H,k", [(1, 2048, 8), (5, 33, 3), (300, 256, 1), (64, 4096, 5), (7, 8200, 64), (2100, 1000, 2), (9, 1111, 9),
                                   (2, 32768, 7)])
@pytest.mark.parametrize("y_type,r_type", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_post_norm_of_rows(B, H, k, y_type, r_type):
    g = gen(B + H + k)
    R = B * k + 5
    y, r = randn(g, R, H).to(TYPES[y_type]), randn(g, B, H).to(TYPES[r_type])
    position = torch.randint(0, R, (B, k), generator=g, device="cuda", dtype=torch.int32)
    w, gain = torch.softmax(randn(g, B, k), 1), 1 + 0.3 * randn(g, H)
    check_post(y, r, quant=H % 32 == 0, post_gain=gain, gain=gain, position=position, topk_w=w, scale=0.5)
    check_post(y, r, gain=gain, gate=a_gate(g, "token", B, H, torch.float32), gate_act="sigmoid", position=position, topk_w=w)
    # the sum is moe_combine's: without a norm of it, gate and scales the block's end is moe_norm of that sum
    out, res, _, _ = md.moe_post_norm(y, r, gain=gain, position=position, topk_w=w, out_dtype=torch.float32)
    o2, res2, _, _ = md.moe_norm(md.moe_combine(y, position, w, out_dtype=torch.float32), gain, residual=r, out_dtype=torch.float32)
    assert torch.equal(bits(res), bits(res2))
    assert ((out - o2).abs() <= (H + 20) * U * o2.abs()).all()
    for bad in (-1, R, 2 ** 31 - 1):
        p2 = position.clone()
        p2[B // 2, k - 1] = bad
        o3, res3, _, _ = md.moe_post_norm(y, r, gain=gain, position=p2, topk_w=w, out_dtype=torch.float32)
        keep = torch.arange(B, device="cuda") != B // 2
        assert o3[B // 2].isnan().all() and res3[B // 2].isnan().all()
        assert torch.equal(bits(o3[keep]), bits(out[keep])) and torch.equal(bits(res3[keep]), bits(res[keep]))


@pytest.mark.parametrize("H", [3, 31, 777, 1111, 4095, 4104, 8195, 20001])
def test_post_norm_reads_and_writes_nothing_behind(H):
    """NaN around the inputs changes nothing; what lies around the outputs stays."""
    g = gen(H)

    def inside(t):
        buf = torch.full((t.numel() + 1024,), float("nan"), device="cuda", dtype=t.dtype)
        buf[512:512 + t.numel()] = t.reshape(-1)
        return buf[512:512 + t.numel()].view(t.shape)

    for dt in TYPES.values():
        y, r, gain, gate = (randn(g, *s).to(dt) for s in ((5, H), (5, H), (H,), (5, H)))
        a = md.moe_post_norm(y, r, post_gain=gain, gate=gate, gain=gain, out_dtype=dt)
        bufs = [torch.full((5 * H + 1024,), 7.0, device="cuda", dtype=dt) for _ in range(2)]
        out, res = (t[512:512 + 5 * H].view(5, H) for t in bufs)
        md.moe_post_norm(inside(y), inside(r), post_gain=inside(gain), gate=inside(gate), gain=inside(gain), out=out, residual_out=res)
        assert torch.equal(bits(out), bits(a[0])) and torch.equal(bits(res), bits(a[1]))
        for t in bufs:
            assert (t[:512] == 7).all() and (t[512 + 5 * H:] == 7).all()


def test_post_norm_past_32_bits():
    """Expert rows, tokens and outputs past 4 GiB."""
    B, H, k = 600000, 4097, 2
    R = B + 7
    y = torch.empty(R, H, device="cuda", dtype=torch.bfloat16)
    for part in y.split(1 << 15):
        part.normal_(generator=gen(3))
    r = torch.empty(B, H, device="cuda", dtype=torch.bfloat16)
    for part in r.split(1 << 15):
        part.normal_(generator=gen(4))
    position = torch.stack([torch.arange(B, device="cuda"), R - 1 - torch.arange(B, device="cuda")], 1).int()
    w, gain = torch.full((B, k), 0.5, device="cuda"), torch.ones(H, device="cuda")
    out, res, _, _ = md.moe_post_norm(y, r, post_gain=gain, gain=gain, position=position, topk_w=w)
    for rows in (slice(0, 3), slice(B - 3, B), slice(524200, 524300)):
        a, b, _, _ = md.moe_post_norm(y[position[rows].long()].flatten(0, 1), r[rows].clone(), post_gain=gain, gain=gain,
                                      position=torch.arange(2 * (rows.stop - rows.start), device="cuda", dtype=torch.int32).view(-1, 2),
                                      topk_w=w[rows].clone())
        n = rows.stop - rows.start
        assert torch.equal(bits(out[rows]), bits(a)) and torch.equal(bits(res[rows]), bits(b)) and n == a.shape[0]


def test_post_norm_in_place():
    g = gen(5)
    for H in (512, 777):
        y, r = randn(g, 9, H).bfloat16(), randn(g, 9, H).bfloat16()
        gain = torch.ones(H, device="cuda")
        out, res, _, _ = md.moe_post_norm(y, r, post_gain=gain, gain=gain, scale=0.5)
        y2, r2 = y.clone(), r.clone()
        o2, res2, _, _ = md.moe_post_norm(y2, r2, post_gain=gain, gain=gain, scale=0.5, out=y2, residual_out=r2)
        assert o2 is y2 and res2 is r2 and torch.equal(bits(y2), bits(out)) and torch.equal(bits(r2), bits(res))
        y3, r3 = y.clone(), r.clone()
        md.moe_post_norm(y3, r3, post_gain=gain, gain=gain, scale=0.5, out=r3, residual_out=y3)
        assert torch.equal(bits(r3), bits(out)) and torch.equal(bits(y3), bits(res))


def test_post_norm_special_values():
    g = gen(6)
    y, r = randn(g, 8, 96), randn(g, 8, 96)
    y[0] = 0.0                                                # a block that adds nothing
    y[1, 3] = float("nan")
    y[2, 40] = float("inf")
    y[3] *= 1e-30                                             # squares underflow: eps stands alone under the root
    r[4] = 0.0
    y[4] = 0.0                                                # nothing at all
    r[5, 50] = float("nan")
    y[6, 70] = 3e19                                           # the square overflows: the normed row is 0
    gain = torch.ones(96, device="cuda")
    out, res, q, s = md.moe_post_norm(y, r, post_gain=gain, gain=gain, out_dtype=torch.float32, quantize=True)
    assert torch.equal(res[0], r[0])
    assert out[1].isnan().all() and res[1].isnan().all() and (s[1] == 255).all()
    assert res[2, 40].isnan() and torch.equal(res[2, :32], r[2, :32]) and out[2].isnan().all()
    assert ((res[3].double() - r[3].double()).abs() <= U * r[3].double().abs() + 1e-26).all()
    assert (out[4] == 0).all() and (res[4] == 0).all()
    assert out[5].isnan().all() and res[5].isnan().sum() == 1
    assert torch.equal(res[6], r[6])
    rq, rs = quantize(out)
    assert torch.equal(s, rs) and torch.equal(q, rq)
    # with eps = 0 tiny rows are exact to rounding, in both norms
    tiny = torch.ldexp(randn(g, 4, 96), torch.tensor([[-140], [-126], [-70], [-45]], device="cuda"))
    out, res, _, _ = md.moe_post_norm(tiny, torch.zeros(4, 96, device="cuda"), post_gain=gain, gain=gain, post_eps=0.0, eps=0.0,
                                      out_dtype=torch.float32)
    ref = tiny.double() / torch.sqrt((tiny.double() ** 2).mean(1, keepdim=True))
    assert ((res.double() - ref).abs() <= 70 * U * ref.abs()).all() and ((out.double() - ref).abs() <= 140 * U * ref.abs()).all()
    out, res, _, _ = md.moe_post_norm(torch.zeros(4, 96, device="cuda"), tiny, gain=gain, eps=0.0, out_dtype=torch.float32)
    assert torch.equal(res, tiny) and ((out.double() - ref).abs() <= 70 * U * ref.abs()).all()


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
def test_post_norm_without_a_gate(act):
    """An activation of no gate has no effect."""
    g = gen(23)
    y, r, gain = randn(g, 5, 320), randn(g, 5, 320), randn(g, 320)
    for a, b in zip(md.moe_post_norm(y, r, gain=gain, scale=0.7, quantize=True),
                    md.moe_post_norm(y, r, gain=gain, scale=0.7, quantize=True, gate_act=act)):
        assert torch.equal(bits(a), bits(b))


def test_post_norm_empty_and_refusals():
    y, r, gain = torch.ones(4, 64, device="cuda"), torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    assert md.moe_post_norm(y[:0], r[:0], gain=gain)[0].shape == (0, 64)
    pos, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.ones(4, 2, device="cuda")
    for kw, err in (({"out": y}, ValueError), ({"quantize": True}, ValueError), ({"gain": gain, "out_dtype": None}, ValueError),
                    ({"gate_act": "silu"}, ValueError), ({"gate": gain, "gate_act": "silu"}, ValueError), ({"gate": w}, ValueError),
                    ({"position": pos}, ValueError), ({"topk_w": w}, ValueError), ({"position": pos[:3], "topk_w": w[:3]}, ValueError),
                    ({"gain": gain, "out_q": y}, ValueError), ({"post_gain": gain[:32]}, ValueError), ({"gain": gain.half()}, TypeError),
                    ({"gain": gain, "out": r, "residual_out": r}, md.MoedError), ({"post_eps": -1.0}, md.MoedError)):
        with pytest.raises(err):
            md.moe_post_norm(y, r, **kw)
    with pytest.raises(ValueError):
        md.moe_post_norm(y[:3], r, gain=gain)
    # no rows at all: every position is bad
    out, res, _, _ = md.moe_post_norm(y[:0], r, gain=gain, position=pos, topk_w=w)
    assert out.isnan().all() and res.isnan().all()


# ---------------------------------------------------------------------------- together

def mx_weights(g, E, N, K):
    q = (randn(g, E, N, K) * 2).to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.randint(118, 121, (E, N, K // 32), generator=g, device="cuda").to(torch.uint8)
    return q, s


def decoded(q, s):
    return q.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).repeat_interleave(32, -1)


class Half:
    """One layer's MoE half: norm, router, experts with a gated shared expert, the norm behind it and the next one's."""

    def __init__(self, B, H=256, E=16, k=4, I=128, seed=1):
        g = gen(seed)
        self.B, self.H, self.E, self.k, self.I = B, H, E, k, I
        self.x, self.r = randn(g, B, H).bfloat16(), randn(g, B, H)
        self.gains = [1 + 0.2 * randn(g, H) for _ in range(3)]
        self.router, self.gate = randn(g, E, H) / math.sqrt(H), randn(g, 1, H).bfloat16() / math.sqrt(H)
        self.bias = 0.05 * randn(g, E)
        self.w = [mx_weights(g, E, I, H), mx_weights(g, E, I, H), mx_weights(g, E, H, I)]

    def run(self, prefill, stream=None):
        s = {"stream": stream}
        n, res, _, _ = md.moe_norm(self.x, self.gains[0], residual=self.r, **s)
        logits = md.moe_linear(n, self.router, out_dtype=torch.float32, **s)
        ids, w = md.moe_route_scored(logits, self.k, bias=self.bias, n_group=4, topk_group=2, routed_scale=1.5, **s)
        gate = md.moe_linear(n, self.gate, activation="sigmoid", out_dtype=torch.float32, **s)
        (gq, gs), (uq, us), (dq, ds) = self.w
        if prefill:
            order, position, offsets = md.moe_group(ids, self.E, **s)
            a = md.moe_grouped_gate_up(n, offsets, gq, gs, uq, us, order=order, k=self.k, **s)
            rows = md.moe_grouped_matmul(a, offsets, dq, ds, out_dtype=torch.float32, **s)
            out = md.moe_post_norm(rows, res, post_gain=self.gains[1], gate=gate, gain=self.gains[2], position=position, topk_w=w, **s)
        else:
            y = md.moe_decode(n, ids, w, gq, gs, uq, us, dq, ds, out_dtype=torch.float32, **s)
            out = md.moe_post_norm(y, res, post_gain=self.gains[1], gate=gate, gain=self.gains[2], **s)
        return n, logits, ids, w, gate, out[0], out[1]

    def reference(self, n, ids, w):
        """From the normed tokens and the router's answer on, in float64."""
        x = n.double()
        gate = torch.sigmoid(x @ self.gate.double().T)
        (wg, wu, wd) = (decoded(*t) for t in self.w)
        y = torch.zeros(self.B, self.H, dtype=torch.float64, device="cuda")
        for j in range(self.k):
            e = ids[:, j].long()
            gt, up = (torch.bmm(t[e], x[:, :, None]).squeeze(-1) for t in (wg, wu))
            y += w[:, j:j + 1].double() * torch.bmm(wd[e], (gt * torch.sigmoid(gt) * up)[:, :, None]).squeeze(-1)
        res = self.x.double() + self.r.double()
        t = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * self.gains[1].double()
        s = res + gate * t
        return gate, s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * self.gains[2].double(), s


@pytest.mark.parametrize("B,prefill", [(1, False), (5, False), (40, True), (300, True)])
def test_half_a_layer(B, prefill):
    h = Half(B)
    n, logits, ids, w, gate, out, s = h.run(prefill)
    check_linear(n, h.router, None, None, None, logits)
    rid, rw = route_ref(logits.cpu().numpy(), h.k, "sigmoid", h.bias.cpu().numpy(), 4, 2, "top2", True, 0, 1.5)
    assert np.array_equal(ids.cpu().numpy(), rid) and np.allclose(w.cpu().numpy(), rw, rtol=2 * U, atol=0)
    rgate, rout, rs = h.reference(n, ids, w)
    assert ((gate.double() - rgate).abs() <= 1e-5).all()
    # the prompt's path rounds the experts' intermediate to bfloat16: 2^-8 of it, in the norm of a row at most; the gate
    # and the norm behind the block keep that relative error, of a part of s
    tol = (2.0 ** -8 if prefill else 1e-4) * 4
    for got, ref in ((s, rs), (out, rout)):
        err = (got.double() - ref).norm(dim=1) / ref.norm(dim=1)
        assert (err <= tol + STEP[got.dtype]).all(), float(err.max())


@pytest.mark.parametrize("B,prefill", [(3, False), (200, True)])
def test_captured_and_replayed(B, prefill):
    """Captured once, replayed on new inputs, with eager work between the replays."""
    h = Half(B, seed=4)
    h.run(prefill)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = h.run(prefill)
    for seed in range(4):
        h.x.copy_(randn(gen(50 + seed), B, h.H))
        want = [t.clone() for t in h.run(prefill)]
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(bits(a), bits(b))
        md.moe_linear(randn(gen(seed), 64, 7168).bfloat16(), randn(gen(9), 256, 7168))


def test_captured_with_one_workspace():
    """Two graphs whose products are split and whose sums lie in the same workspace, replayed in turn."""
    types = (torch.bfloat16, torch.float32)
    sizes = [(64, 7168, 256), (700, 4096, 900)]
    need = [md.moe_linear_workspace_bytes(*size, *types) for size in sizes]
    assert min(need) > 0
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    calls = []
    for i, (B, K, N) in enumerate(sizes):
        g = gen(60 + i)
        calls.append([randn(g, B, K).bfloat16(), randn(g, N, K), randn(g, B, N), torch.empty(B, N, device="cuda")])
    graphs = []
    for x, w, r, out in calls:
        md.moe_linear(x, w, residual=r, activation="tanh", out=out, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            md.moe_linear(x, w, residual=r, activation="tanh", out=out, workspace=ws)
    for rep in range(3):
        for i, (x, w, r, out) in enumerate(calls):
            x.copy_(randn(gen(70 + 2 * rep + i), *x.shape))
            out.fill_(float("nan"))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for x, w, r, out in calls:
            assert torch.equal(bits(out), bits(md.moe_linear(x, w, residual=r, activation="tanh", out_dtype=torch.float32)))


def test_two_streams():
    """Calls on streams of their own, handed over as stream or as a raw handle; results made by the call."""
    halves = [Half(64, seed=7), Half(64, seed=8)]
    want = [[t.clone() for t in h.run(True)] for h in halves]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for rep in range(3):
        got = [h.run(True, stream=s if rep % 2 else s.cuda_stream) for h, s in zip(halves, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for t, u in zip(a, b):
                assert torch.equal(bits(t), bits(u))
