"""The prompt-side operators of the MoE block: what is timed, in elementary torch and through the library.

A decode step takes a few tokens through `moe_decode`. A prompt brings thousands of tokens at once, and the
block around the experts becomes five operators:

* norm     -- residual addition and root-mean-square norm in front of the router and the experts, with the
              result in bfloat16 and, beside it, in MXFP8 (E4M3 codes, one UE8M0 scale per 32 values);
* group    -- the routed slots sorted by expert (stable), with their offsets and positions;
* gate_up  -- SiLU(x Wg^T) * (x Wu^T) over the rows of each expert, ragged, rows gathered by token;
* matmul   -- the product with one matrix per expert over ragged rows (the down projection);
* combine  -- each token's k expert rows summed with its routing weights.

Weights are MXFP8 or MXFP4, activations bfloat16 or MXFP8, sums float32. `own` chooses between the plain
form and the library.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------- cases

def _norm(name, B, H, x="bf16", residual="bf16", out="bf16", mx=False):
    return {"name": name, "op": "norm", "B": B, "H": H, "x": x, "residual": residual, "out": out, "mx": mx}


def _group(name, B, E, k, zipf=0.0):
    return {"name": name, "op": "group", "B": B, "E": E, "k": k, "zipf": zipf}


def _product(name, op, B, E, k, K, N, act, w, out, zipf=0.0):
    return {"name": name, "op": op, "B": B, "E": E, "k": k, "K": K, "N": N, "act": act, "w": w, "out": out,
            "zipf": zipf}


def _combine(name, B, k, H, y="bf16", out="bf16"):
    return {"name": name, "op": "combine", "B": B, "k": k, "H": H, "y": y, "out": out}


def listed():
    return [
        # one decode token in front of the router: latency
        _norm("norm token", 1, 2048),
        # a float32 residual stream, rows of no power of two, a mid-sized batch
        _norm("norm odd f32", 333, 1111, x="f32", residual="f32", out="f32"),
        # a long prompt: bfloat16 for the router, MXFP8 for the experts
        _norm("norm prompt mx", 8192, 4096, mx=True),
        # a decode batch whose routing is skewed
        _group("group batch", 64, 256, 8, zipf=1.1),
        # a long prompt's routing
        _group("group prompt", 16384, 128, 8),
        # a few tokens: nearly every routed expert has a single row, and reading the weights is all
        _product("gate_up few", "gate_up", 8, 128, 8, 2048, 768, "bf16", "mxfp8", "bf16"),
        # a chunk of a prompt, MXFP4 weights, row counts of no tile's multiple
        _product("gate_up chunk fp4", "gate_up", 1000, 128, 8, 2048, 768, "bf16", "mxfp4", "bf16"),
        # a long prompt all in eight bits: the intermediate leaves as MXFP8 for the down projection
        _product("gate_up prompt mx", "gate_up", 8192, 128, 8, 2048, 768, "mxfp8", "mxfp8", "mxfp8"),
        # long rows, skewed routing: some experts with most of the tokens, some with none
        _product("matmul skewed", "matmul", 1024, 256, 8, 2048, 7168, "bf16", "mxfp8", "f32", zipf=1.1),
        # the down projection of the long prompt
        _product("matmul prompt mx", "matmul", 8192, 128, 8, 768, 2048, "mxfp8", "mxfp8", "bf16"),
        # one decode token, float32 rows
        _combine("combine token", 1, 8, 2048, y="f32"),
        # the long prompt
        _combine("combine prompt", 8192, 8, 2048),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "group", "gate_up", "gate_up", "matmul", "matmul", "combine"))
    t = ("bf16", "f32")
    if op == "norm":
        mx = rng.random() < 0.4
        H = 32 * _log(rng, 8, 224) if mx else _log(rng, 200, 7168)
        return _unnamed(_norm("", _log(rng, 1, max(1, 8192 * 4096 // H)), H, x=rng.choice(t),
                              residual=rng.choice(t + ("none",)), out=rng.choice(t), mx=mx))
    E = _log(rng, 8, 256)
    k = rng.randint(1, 8)
    zipf = rng.choice((0.0, 0.0, 1.1))
    if op == "group":
        return _unnamed(_group("", _log(rng, 1, 16384), E, k, zipf))
    if op == "combine":
        H = _log(rng, 200, 7168)
        return _unnamed(_combine("", _log(rng, 1, max(1, 8192 * 8 * 2048 // (H * k))), k, H, y=rng.choice(t),
                                 out=rng.choice(t)))
    K = 32 * _log(rng, 4, 224)
    N = 32 * _log(rng, 4, 224 if op == "matmul" else 64)
    # no more work, and no more weights, than the largest listed case
    while E * K * N * (2 if op == "gate_up" else 1) > 256 * 2048 * 7168:
        E //= 2
    E = max(E, k)
    most = 8192 * 8 * 2048 * 768 // (K * N * k)
    return _unnamed(_product("", op, _log(rng, 1, max(1, min(8192, most))), E, k, K, N, rng.choice(("bf16", "mxfp8")),
                             rng.choice(("mxfp8", "mxfp4")),
                             rng.choice(("bf16", "f32") if op == "matmul" else ("bf16", "f32", "mxfp8")), zipf))


def _unnamed(case):
    del case["name"]
    return case


# ---------------------------------------------------------------------------- work

_BYTES = {"bf16": 2.0, "f32": 4.0, "none": 0.0, "mxfp8": 33 / 32, "mxfp4": 17 / 32}


def _touched(B, E, k, zipf):
    """Experts with at least one row, by the share of tokens that take each (a sample's, where it is skewed)."""
    if not zipf:
        return E * (1 - (1 - k / E) ** B)
    logits = np.random.RandomState(0).standard_normal((2048, E)) - zipf * np.log(np.arange(1, E + 1))
    top = np.argpartition(-logits, k - 1, axis=1)[:, :k] if k < E else np.tile(np.arange(E), (2048, 1))
    return float(np.sum(1 - (1 - np.bincount(top.reshape(-1), minlength=E) / 2048) ** B))


def work(case):
    op, B = case["op"], case["B"]
    if op == "norm":
        n = B * case["H"]
        b = _BYTES[case["x"]] + 2 * _BYTES[case["residual"]] + _BYTES[case["out"]] + (_BYTES["mxfp8"] if case["mx"] else 0)
        return {"bytes": n * b + 4 * case["H"], "flops": 5 * n}
    if op == "group":
        n = B * case["k"]
        return {"bytes": 12 * n + 4 * (case["E"] + 1), "flops": n}
    k = case["k"]
    if op == "combine":
        n = B * case["H"]
        return {"bytes": n * (k * _BYTES[case["y"]] + _BYTES[case["out"]]) + 8 * B * k, "flops": 2 * n * k}
    E, K, N = case["E"], case["K"], case["N"]
    two = 2 if op == "gate_up" else 1
    touched = _touched(B, E, k, case["zipf"])
    rows = B if op == "gate_up" else B * k
    return {"bytes": touched * two * N * K * _BYTES[case["w"]] + rows * K * _BYTES[case["act"]] +
            B * k * N * _BYTES[case["out"]] + 4 * (B * k + E + 1),
            "flops": 2.0 * two * B * k * N * K}


# ---------------------------------------------------------------------------- inputs

_T = {"bf16": torch.bfloat16, "f32": torch.float32}


def _to_mx8(v):
    """Float32 [..., K] -> E4M3 codes [..., K] and UE8M0 scale codes [..., K/32], both uint8."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 9).clamp(-127, 127)          # floor(log2 amax) - 8
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    q = torch.ldexp(b, -e).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    s = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8).squeeze(-1)
    q = torch.where(bad, torch.full_like(q, 0x7F), q)
    return q.reshape(v.shape), s


def _to_mx4(v):
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 3).clamp(-127, 127), -127)
    t = torch.ldexp(b, -e)
    m = t.abs().clamp(max=6)
    # nearest of 0 0.5 1 1.5 2 3 4 6: steps of 0.5 below 2, of 1 below 4, of 2 above
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    r = torch.round(m / step) * step
    c = torch.searchsorted(torch.tensor(E2M1, device=v.device), r).to(torch.uint8)
    c = (c | ((t < 0).to(torch.uint8) << 3)).reshape(*v.shape[:-1], v.shape[-1] // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), (e + 127).to(torch.uint8).squeeze(-1)


def _routing(g, B, E, k, zipf):
    logits = torch.randn((B, E), generator=g, device="cuda")
    if zipf:
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        logits = logits - zipf * torch.log(rank.float())
    top = torch.topk(logits, k, dim=1)
    return top.indices.to(torch.int32), torch.softmax(top.values, 1)


def _grouped(ids, E):
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=ids.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum((flat[:, None] == torch.arange(E, device=ids.device)).sum(0), 0)
    return order.to(torch.int32), position.to(torch.int32).reshape(ids.shape), offsets.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s, op, B = dict(case), case["op"], case["B"]
    if op == "norm":
        H = case["H"]
        s["xv"] = rand(B, H).to(_T[case["x"]])
        s["rv"] = None if case["residual"] == "none" else (rand(B, H) * 3).to(_T[case["residual"]])
        s["gain"] = (1 + 0.2 * rand(H)).to(torch.bfloat16)
        return s
    if op == "combine":
        R = B * case["k"]
        s["yv"] = rand(R, case["H"]).to(_T[case["y"]])
        s["position"] = torch.randperm(R, generator=g, device="cuda").to(torch.int32).reshape(B, case["k"])
        s["weight"] = torch.softmax(rand(B, case["k"]), 1)
        return s
    ids, _ = _routing(g, B, case["E"], case["k"], case["zipf"])
    if op == "group":
        s["ids"] = ids
        return s
    E, k, K, N = case["E"], case["k"], case["K"], case["N"]
    s["order"], _, s["offsets"] = _grouped(ids, E)
    v = rand(B if op == "gate_up" else B * k, K)
    s["a"], s["a_s"] = _to_mx8(v) if case["act"] == "mxfp8" else (v.to(torch.bfloat16), None)
    # weights of a trained layer's spread, encoded along K some experts at a time
    encode, kb = (_to_mx4, K // 2) if case["w"] == "mxfp4" else (_to_mx8, K)
    for name in ("w", "u") if op == "gate_up" else ("w",):
        s[name + "_q"] = torch.empty((E, N, kb), dtype=torch.uint8, device="cuda")
        s[name + "_s"] = torch.empty((E, N, K // 32), dtype=torch.uint8, device="cuda")
        for some in torch.arange(E).split(max(1, (1 << 28) // (N * K))):
            i, j = int(some[0]), int(some[-1]) + 1
            s[name + "_q"][i:j], s[name + "_s"][i:j] = encode(rand(j - i, N, K) * 0.02)
    return s


# ---------------------------------------------------------------------------- one pass

def _decoded(q, scale, fmt):
    """Codes and scales -> float32 values."""
    if fmt == "mxfp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
        v = table[torch.stack((q & 15, q >> 4), -1).long()].reshape(*q.shape[:-1], 2 * q.shape[-1])
    else:
        v = q.view(torch.float8_e4m3fn).float()
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    return torch.ldexp(b, scale[..., None].int() - 127).reshape(v.shape)


def _mx_values(q, s):
    """Codes and scales as the numbers that they stand for."""
    return q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)


def _by_expert(rows, offsets):
    """Sorted rows [R, K] -> [E, most, K] (zeros behind each expert's last row), and each row's place in it."""
    E, R = offsets.numel() - 1, rows.shape[0]
    most = max(1, int((offsets[1:] - offsets[:-1]).max()))
    at = torch.arange(R, device=rows.device)
    e = torch.searchsorted(offsets[1:].long(), at, right=True)
    place = e * most + at - offsets[e].long()
    x = torch.zeros((E * most, rows.shape[1]), device=rows.device)
    x[place] = rows
    return x.view(E, most, -1), place


def _products(rows, place, q, scale, fmt):
    return torch.bmm(rows, _decoded(q, scale, fmt).transpose(1, 2)).flatten(0, 1)[place]


def run(s):
    op = s["op"]
    if own:
        from output_centric_expert_amd import moedecode as md
        if op == "norm":
            out, res, q, sc = md.moe_norm(s["xv"], s["gain"], residual=s["rv"], eps=EPS, out_dtype=_T[s["out"]],
                                          quantize=s["mx"])
            return [v for v in (out, res) if v is not None] + (list(_mx_values(q, sc)) if s["mx"] else [])
        if op == "group":
            return md.moe_group(s["ids"], s["E"])
        if op == "combine":
            return md.moe_combine(s["yv"], s["position"], s["weight"], out_dtype=_T[s["out"]])
        if op == "gate_up":
            mx = s["out"] == "mxfp8"
            r = md.moe_grouped_gate_up(s["a"], s["offsets"], s["w_q"], s["w_s"], s["u_q"], s["u_s"], order=s["order"],
                                       k=s["k"], a_s=s["a_s"], out_dtype=torch.bfloat16 if mx else _T[s["out"]],
                                       quantize=mx, wformat=s["w"])
            return _mx_values(*r) if mx else r
        return md.moe_grouped_matmul(s["a"], s["offsets"], s["w_q"], s["w_s"], a_s=s["a_s"], out_dtype=_T[s["out"]],
                                     wformat=s["w"])
    if op == "norm":
        v = s["xv"].float()
        res = None
        if s["rv"] is not None:
            v = v + s["rv"].float()
            res = v.to(s["rv"].dtype)
        y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["gain"].float()
        outs = [y.to(_T[s["out"]])] + ([] if res is None else [res])
        return outs + (list(_mx_values(*_to_mx8(y))) if s["mx"] else [])
    if op == "group":
        return _grouped(s["ids"], s["E"])
    if op == "combine":
        rows = s["yv"][s["position"].long()].float()
        return (rows * s["weight"][..., None]).sum(1).to(_T[s["out"]])
    a = s["a"].float() if s["a_s"] is None else _decoded(s["a"], s["a_s"], "mxfp8")
    if op == "matmul":
        rows, place = _by_expert(a, s["offsets"])
        return _products(rows, place, s["w_q"], s["w_s"], s["w"]).to(_T[s["out"]])
    rows, place = _by_expert(a[s["order"].long() // s["k"]], s["offsets"])
    gate = _products(rows, place, s["w_q"], s["w_s"], s["w"])
    y = gate / (1 + torch.exp(-gate)) * _products(rows, place, s["u_q"], s["u_s"], s["w"])
    return _mx_values(*_to_mx8(y)) if s["out"] == "mxfp8" else y.to(_T[s["out"]])


# ---------------------------------------------------------------------------- 64 bits

def _values64(q, scale, fmt):
    """Float64 values of MX codes from the formats' bit fields."""
    if fmt == "mxfp4":
        c = torch.stack((q & 15, q >> 4), -1).flatten(-2).to(torch.int32)
        exp, man, sign, bias, bits = (c >> 1) & 3, c & 1, c >> 3, 1, 1
    else:
        c = q.to(torch.int32)
        exp, man, sign, bias, bits = (c >> 3) & 15, c & 7, c >> 7, 7, 3
    frac = man.double() / (1 << bits)
    v = torch.where(exp > 0, 1 + frac, frac) * torch.exp2((exp.clamp(min=1) - bias).double())
    if fmt != "mxfp4":
        v = torch.where((c & 127) == 127, float("nan"), v)
    v = torch.where(sign > 0, -v, v)
    return v * torch.exp2(scale.double() - 127).repeat_interleave(32, -1)


def _mx64(v):
    """Float64 [..., K] -> the values of its E4M3 codes and of its block scales."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    two = torch.exp2(torch.floor(torch.log2(amax.clamp(min=2.0 ** -200))) - 8).clamp(2.0 ** -127, 2.0 ** 127)
    two = torch.where(amax == 0, 2.0 ** -127, two)
    t = (b / two).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(t / step) * step).flatten(-2), two.squeeze(-1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        v = s["xv"].double() if s["rv"] is None else s["xv"].double() + s["rv"].double()
        y = v / torch.sqrt(torch.sum(v ** 2, 1, keepdim=True) / case["H"] + EPS) * s["gain"].double()
        return [y] + ([] if s["rv"] is None else [v]) + (list(_mx64(y)) if case["mx"] else [])
    if op == "group":
        ids = s["ids"].cpu().numpy().reshape(-1)
        order = np.lexsort((np.arange(ids.size), ids))
        position = np.zeros(ids.size, np.int64)
        position[order] = np.arange(ids.size)
        offsets = np.concatenate([[0], np.cumsum(np.bincount(ids, minlength=case["E"]))])
        return order, position.reshape(s["ids"].shape), offsets
    if op == "combine":
        out = torch.zeros((case["B"], case["H"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            out += s["yv"].index_select(0, s["position"][:, j].long()).double() * s["weight"][:, j:j + 1].double()
        return out
    a = s["a"].double() if s["a_s"] is None else _values64(s["a"], s["a_s"], "mxfp8")
    ends = s["offsets"].tolist()
    out = torch.empty((ends[-1], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        if op == "matmul":
            out[lo:hi] = a[lo:hi] @ _values64(s["w_q"][e], s["w_s"][e], case["w"]).T
        else:
            x = a[torch.div(s["order"][lo:hi], case["k"], rounding_mode="floor").long()]
            gate = x @ _values64(s["w_q"][e], s["w_s"][e], case["w"]).T
            out[lo:hi] = gate * torch.sigmoid(gate) * (x @ _values64(s["u_q"][e], s["u_s"][e], case["w"]).T)
    return _mx64(out) if case["out"] == "mxfp8" else out
