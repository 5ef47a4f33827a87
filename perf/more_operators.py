"""The operators around the MoE block: what is timed, in elementary torch and through the library.

* linear -- a dense product with bias, activation and residual: router logits, gates, dense layers;
* route  -- the router's choice from its logits: softmax or sigmoid scores, a bias for balance, groups of experts,
            top-k, renormalised weights;
* post   -- the end of a block: the norm of its output (given, or summed from the experts' rows), gate, scales,
            residual, and the norm in front of the next block, with the result in MXFP8 too.

Activations and weights are bfloat16 or float32, sums float32. `own` chooses between the plain form and the library.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
_T = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases

def _linear(name, B, K, N, x="bf16", w="bf16", out="bf16", bias=False, act="none", residual="none"):
    return {"name": name, "op": "linear", "B": B, "K": K, "N": N, "x": x, "w": w, "out": out, "bias": bias, "act": act,
            "residual": residual}


def _route(name, B, E, k, score="sigmoid", logits="f32", bias=True, groups=1, take=1, group_score="top2", renorm=True,
           shared=0):
    return {"name": name, "op": "route", "B": B, "E": E, "k": k, "score": score, "logits": logits, "bias": bias,
            "groups": groups, "take": take, "group_score": group_score, "renorm": renorm, "shared": shared}


def _post(name, B, H, k=0, y="bf16", residual="bf16", out="bf16", post=True, gate="none", gate_act="none", mx=False):
    return {"name": name, "op": "post", "B": B, "H": H, "k": k, "y": y, "residual": residual, "out": out, "post": post,
            "gate": gate, "gate_act": gate_act, "mx": mx}


def listed():
    return [
        # the router's logits of one decode token: latency
        _linear("router token", 1, 2048, 128, w="f32", out="f32"),
        # the router's logits of a decode batch, long rows
        _linear("router batch", 64, 7168, 256, w="f32", out="f32"),
        # the router's logits of a long prompt
        _linear("router prompt", 8192, 7168, 256, w="f32", out="f32"),
        # a projection of a decode batch with the residual added: reading the weights is all
        _linear("projection batch", 32, 4096, 4096, bias=True, residual="bf16"),
        # a dense layer of a long prompt
        _linear("dense prompt", 8192, 4096, 4096, bias=True, act="silu", residual="bf16"),
        # a chunk of a prompt in float32, sizes of no tile's multiple
        _linear("chunk odd f32", 1000, 1111, 777, x="f32", w="f32", out="f32", bias=True, act="gelu", residual="f32"),
        # one decode token: softmax scores, no groups
        _route("route token", 1, 128, 8, score="softmax", bias=False),
        # a decode batch: sigmoid scores, bias, 4 of 8 groups, a shared expert
        _route("route batch", 64, 256, 8, groups=8, take=4, shared=1),
        # a long prompt
        _route("route prompt", 16384, 256, 8, groups=8, take=4),
        # the end of the block of one decode token, a gate per token
        _post("post token", 1, 2048, gate="token", gate_act="sigmoid"),
        # a long prompt: the block's output with a gate per channel, MXFP8 for the experts of the next layer
        _post("post prompt mx", 8192, 4096, gate="channel", mx=True),
        # a long prompt, straight from the experts' rows, float32 residual stream
        _post("post rows prompt", 8192, 2048, k=8, residual="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear", "route", "route", "post", "post"))
    t = ("bf16", "f32")
    if op == "linear":
        K, N = _log(rng, 32, 7168), _log(rng, 1, 7168)
        if rng.random() < 0.5:
            K = 32 * max(1, K // 32)
        x, w = rng.choice(("bf16", "bf16", "f32")), rng.choice(t)
        products = (1 if x == w == "bf16" else 6 if x == w else 3)
        most = min(8192, 8192 * 4096 * 4096 // (K * N * products))
        # no more bytes than the largest listed case
        most = min(most, 8192 * 4096 * 3 // (K + 2 * N) // (2 if "f32" in (x, w) else 1))
        return _unnamed(_linear("", _log(rng, 1, max(1, most)), K, N, x=x, w=w, out=rng.choice(t), bias=rng.random() < 0.5,
                                act=rng.choice(("none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid")),
                                residual=rng.choice(("none",) + t)))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 5, 8))
        E = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        take = rng.randint(1, groups)
        k = rng.randint(1, min(8, take * (E // groups)))
        return _unnamed(_route("", _log(rng, 1, 16384 * 256 // max(E, 256)), E, k, score=rng.choice(("sigmoid", "softmax")),
                               logits=rng.choice(t), bias=rng.random() < 0.6, groups=groups, take=take,
                               group_score=rng.choice(("top2", "max")), renorm=rng.random() < 0.7, shared=rng.choice((0, 0, 1, 2))))
    mx = rng.random() < 0.4
    H = 32 * _log(rng, 8, 224) if mx else _log(rng, 200, 7168)
    k = rng.choice((0, 0, rng.randint(1, 8)))
    most = 8192 * 2048 * 8 // (H * k) if k else 8192 * 4096 // H
    return _unnamed(_post("", _log(rng, 1, max(1, min(8192, most))), H, k=k, y=rng.choice(t), residual=rng.choice(t),
                          out=rng.choice(t), post=rng.random() < 0.7,
                          gate=rng.choice(("none", "token", "channel", "full")), gate_act=rng.choice(("none", "sigmoid", "tanh")),
                          mx=mx))


def _unnamed(case):
    del case["name"]
    return case


# ---------------------------------------------------------------------------- work

_BYTES = {"bf16": 2.0, "f32": 4.0, "none": 0.0, "mxfp8": 33 / 32}


def work(case):
    op, B = case["op"], case["B"]
    if op == "linear":
        K, N = case["K"], case["N"]
        return {"bytes": B * K * _BYTES[case["x"]] + N * K * _BYTES[case["w"]] + (4 * N if case["bias"] else 0) +
                B * N * (_BYTES[case["residual"]] + _BYTES[case["out"]]), "flops": 2.0 * B * K * N}
    if op == "route":
        E = case["E"]
        return {"bytes": B * E * _BYTES[case["logits"]] + (4 * E if case["bias"] else 0) +
                8 * B * (case["k"] + case["shared"]), "flops": 10.0 * B * E}
    H, k = case["H"], case["k"]
    gate = {"none": 0, "token": B, "channel": H, "full": B * H}[case["gate"]]
    b = B * H * (max(k, 1) * _BYTES[case["y"]] + 2 * _BYTES[case["residual"]] + _BYTES[case["out"]] +
                 (_BYTES["mxfp8"] if case["mx"] else 0))
    return {"bytes": b + 8 * B * k + 2 * gate + 4 * H, "flops": 2.0 * B * H * (5 + k)}


# ---------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s, op, B = dict(case), case["op"], case["B"]
    if op == "linear":
        K, N = case["K"], case["N"]
        # normed activations, weights of a trained layer's spread
        s["xv"] = (rand(B, K) * (1 + 0.2 * rand(K))).to(_T[case["x"]])
        s["wv"] = (rand(N, K) / math.sqrt(K)).to(_T[case["w"]])
        s["bv"] = 0.5 * rand(N) if case["bias"] else None
        s["rv"] = None if case["residual"] == "none" else (2 * rand(B, N)).to(_T[case["residual"]])
        return s
    if op == "route":
        E = case["E"]
        # some experts are more popular than others; the bias works against it
        liked = rand(E)
        s["lv"] = (1.5 * rand(B, E) + 0.5 * liked).to(_T[case["logits"]])
        s["bv"] = -0.1 * liked + 0.02 * rand(E) if case["bias"] else None
        return s
    H, k = case["H"], case["k"]
    s["yv"] = rand(B * max(k, 1), H).to(_T[case["y"]])
    s["position"] = torch.randperm(B * k, generator=g, device="cuda").to(torch.int32).reshape(B, k) if k else None
    s["weight"] = torch.softmax(rand(B, k), 1) if k else None
    s["rv"] = (3 * rand(B, H)).to(_T[case["residual"]])
    s["post_gain"] = (1 + 0.2 * rand(H)).to(torch.bfloat16) if case["post"] else None
    shape = {"none": None, "token": (B, 1), "channel": (H,), "full": (B, H)}[case["gate"]]
    s["gate_v"] = None if shape is None else rand(*shape).to(torch.bfloat16)
    s["gain"] = (1 + 0.2 * rand(H)).to(torch.bfloat16)
    return s


SCALE, RESIDUAL_SCALE = 0.7, 0.9                 # of the block's output and of the residual
ROUTED_SCALE = 2.5


# ---------------------------------------------------------------------------- one pass

def _to_mx8(v):
    """Float32 [..., K] as the values of its E4M3 codes and of its UE8M0 scales, one for 32 values."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 9).clamp(-127, 127), -127)     # floor(log2 amax) - 8
    q = torch.ldexp(b, -e).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.flatten(-2), (e + 127).to(torch.uint8).squeeze(-1).view(torch.float8_e8m0fnu)


def _activated(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "relu":
        return torch.clamp(v, min=0)
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    if act == "tanh":
        return torch.tanh(v)
    return v


def _named(act):
    return None if act == "none" else act


def run(s):
    op = s["op"]
    if own:
        from output_centric_expert_amd import moedecode as md
        if op == "linear":
            return md.moe_linear(s["xv"], s["wv"], bias=s["bv"], activation=_named(s["act"]), residual=s["rv"],
                                 out_dtype=_T[s["out"]])
        if op == "route":
            return md.moe_route_scored(s["lv"], s["k"], score=s["score"], bias=s["bv"], n_group=s["groups"],
                                       topk_group=s["take"], group_score=s["group_score"], renormalize=s["renorm"],
                                       n_shared=s["shared"], routed_scale=ROUTED_SCALE)
        out, res, q, sc = md.moe_post_norm(s["yv"], s["rv"], post_gain=s["post_gain"], post_eps=EPS, gate=s["gate_v"],
                                           gate_act=_named(s["gate_act"]), scale=SCALE, residual_scale=RESIDUAL_SCALE,
                                           gain=s["gain"], eps=EPS, position=s["position"], topk_w=s["weight"],
                                           out_dtype=_T[s["out"]], quantize=s["mx"])
        return [out, res] + ([q.view(torch.float8_e4m3fn), sc.view(torch.float8_e8m0fnu)] if s["mx"] else [])
    if op == "linear":
        v = s["xv"].float() @ s["wv"].float().T
        if s["bv"] is not None:
            v = v + s["bv"]
        v = _activated(v, s["act"])
        return (v if s["rv"] is None else v + s["rv"].float()).to(_T[s["out"]])
    if op == "route":
        return _routed(s)
    y = s["yv"].float()
    if s["position"] is not None:
        y = (y[s["position"].long()] * s["weight"][..., None]).sum(1)
    if s["post_gain"] is not None:
        y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["post_gain"].float()
    if s["gate_v"] is not None:
        y = y * _activated(s["gate_v"].float(), s["gate_act"])
    res = RESIDUAL_SCALE * s["rv"].float() + SCALE * y
    out = res * torch.rsqrt((res * res).mean(1, keepdim=True) + EPS) * s["gain"].float()
    return [out.to(_T[s["out"]]), res.to(s["rv"].dtype)] + (list(_to_mx8(out)) if s["mx"] else [])


def _routed(s):
    """ids int32 and weights float32 [B, k + shared]. A score is rounded to float32 before it is compared, and so is its
    sum with the bias: equal ones go to the lower expert. They are computed in 64 bits, so that the rounded values do not
    depend on the way."""
    E, k, G = s["E"], s["k"], s["groups"]
    logit = s["lv"].double()
    if s["score"] == "softmax":
        e = torch.exp(logit - logit.amax(1, keepdim=True))
        score = (e / e.sum(1, keepdim=True)).float()
    else:
        score = (1 / (1 + torch.exp(-logit))).float()
    choice = score if s["bv"] is None else score + s["bv"]
    if s["take"] < G:
        best = torch.sort(choice.unflatten(1, (G, E // G)), dim=2, descending=True).values
        value = best[..., 0] + best[..., 1] if s["group_score"] == "top2" and E > G else best[..., 0]
        taken = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :s["take"]]
        inside = torch.zeros_like(value, dtype=torch.bool).scatter_(1, taken, True)
        choice = choice.masked_fill(~inside.repeat_interleave(E // G, 1), float("-inf"))
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(score, 1, ids)
    if s["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    shared = torch.arange(E, E + s["shared"], device=ids.device).expand(ids.shape[0], -1)
    return (torch.cat((ids, shared), 1).to(torch.int32),
            torch.cat((w * ROUTED_SCALE, torch.ones_like(shared, dtype=torch.float32)), 1))


# ---------------------------------------------------------------------------- 64 bits

def _mx64(v):
    """Float64 [..., K] -> the values of its E4M3 codes and of its block scales."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    two = torch.exp2(torch.floor(torch.log2(amax.clamp(min=2.0 ** -200))) - 8).clamp(2.0 ** -127, 2.0 ** 127)
    two = torch.where(amax == 0, 2.0 ** -127, two)
    t = (b / two).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(t / step) * step).flatten(-2), two.squeeze(-1)


def _act64(v, act):
    F = torch.nn.functional
    if act == "tanh":
        return torch.tanh(v)
    return {"none": lambda t: t, "silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda t: F.gelu(t, approximate="tanh"),
            "relu": torch.relu, "sigmoid": torch.sigmoid}[act](v)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "linear":
        v = torch.empty((case["B"], case["N"]), dtype=torch.float64, device="cuda")
        w = s["wv"].double()
        for rows in torch.arange(case["B"], device="cuda").split(1024):
            v[rows] = s["xv"][rows].double() @ w.T
        if s["bv"] is not None:
            v += s["bv"].double()
        v = _act64(v, case["act"])
        return v if s["rv"] is None else v + s["rv"].double()
    if op == "route":
        return _exact_route(case, s)
    y = s["yv"].double()
    if case["k"]:
        rows, y = y, torch.zeros((case["B"], case["H"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            y += rows.index_select(0, s["position"][:, j].long()) * s["weight"][:, j:j + 1].double()
    if case["post"]:
        y = y / torch.sqrt(torch.sum(y ** 2, 1, keepdim=True) / case["H"] + EPS) * s["post_gain"].double()
    if case["gate"] != "none":
        y = y * _act64(s["gate_v"].double(), case["gate_act"])
    v = s["rv"].double() * RESIDUAL_SCALE + y * SCALE
    out = v / torch.sqrt(torch.sum(v ** 2, 1, keepdim=True) / case["H"] + EPS) * s["gain"].double()
    return [out, v] + (list(_mx64(out)) if case["mx"] else [])


def _exact_route(case, s):
    B, E, k, G = case["B"], case["E"], case["k"], case["groups"]
    x = s["lv"].double().cpu().numpy()
    if case["score"] == "softmax":
        e = np.exp(x - x.max(1, keepdims=True))
        score = (e / e.sum(1, keepdims=True)).astype(np.float32)
    else:
        score = (1 / (1 + np.exp(-x))).astype(np.float32)
    choice = score if s["bv"] is None else score + s["bv"].cpu().numpy()
    grouped = choice.reshape(B, G, E // G)
    value = grouped.max(2)
    if case["group_score"] == "top2" and E > G:
        value = value + np.partition(grouped, E // G - 2, axis=2)[:, :, E // G - 2]
    order = np.argsort(-value, axis=1, kind="stable")[:, :case["take"]]
    closed = np.ones((B, G), bool)
    np.put_along_axis(closed, order, False, 1)
    choice = np.where(np.repeat(closed, E // G, axis=1), -np.inf, choice)
    ids = np.argsort(-choice, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(score, ids, 1).astype(np.float64)
    if case["renorm"]:
        w /= w.sum(1, keepdims=True) + 1e-20
    shared = np.broadcast_to(np.arange(E, E + case["shared"]), (B, case["shared"]))
    return np.concatenate([ids, shared], 1), np.concatenate([w * ROUTED_SCALE, np.ones(shared.shape)], 1)
