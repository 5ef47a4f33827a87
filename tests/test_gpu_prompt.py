"""GPU tests of the prompt-side operators (moe_norm, moe_group, moe_grouped_gate_up, moe_grouped_matmul,
moe_combine, moe_prefill) against plain float64 computations.

Products are tested two ways: with codes of small whole numbers and power-of-two scales, for which every
float32 sum is exact and the result has to be equal bit for bit (whatever tile, split or order a size takes),
and with quantized normal values against the bound of a float32 sum: n terms in any order are off by at most
n * 2^-24 * sum |terms| to first order; the matrix instructions may truncate where an addition would round, so
2^-23 per term is allowed. A store to bfloat16 is off by at most 2^-8 of the value (half a step)."""
import ctypes

import numpy as np
import pytest
import torch

from output_centric_expert_amd import moedecode as md

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = torch.finfo(torch.bfloat16).eps / 2
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    md.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def decode(q, s, fmt="mxfp8"):
    """Codes and scales -> float64 values."""
    if fmt == "mxfp4":
        v = E2M1.to(q.device)[torch.stack((q & 15, q >> 4), -1).flatten(-2).long()]
    else:
        v = q.view(torch.float8_e4m3fn).double()
    two = torch.exp2(s.double() - 127)
    two[s == 255] = float("nan")
    return v * two.repeat_interleave(32, -1)


def quantize(y):
    """Float32 [..., K] -> codes and scales by the rule of moe_norm, from the bits."""
    b = y.unflatten(-1, (-1, 32))
    field = (b.abs().view(torch.int32).amax(-1)) >> 23
    scale = torch.where(field == 255, torch.full_like(field, 255), (field - 8).clamp(min=0))
    t = torch.ldexp(b.double(), (127 - scale)[..., None].double()).clamp(-448, 448)
    q = t.float().to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.where((scale == 255)[..., None], torch.full_like(q, 0x7F), q)
    return q.flatten(-2), scale.to(torch.uint8)


def random_mx(g, shape, fmt, spread=1.0):
    v = torch.randn(shape, generator=g, device="cuda") * spread
    if fmt == "mxfp8":
        return quantize(v)
    q = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(118, 124, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda", dtype=torch.uint8)
    return q, s


def whole_mx(g, shape, fmt):
    """Codes of whole numbers -2..2 and block scales 1, 2, 4: exact sums."""
    v = torch.randint(-2, 3, shape, generator=g, device="cuda")
    s = torch.randint(127, 130, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda").to(torch.uint8)
    if fmt == "mxfp8":
        return v.float().to(torch.float8_e4m3fn).view(torch.uint8), s
    code = torch.tensor([4, 2, 0, 2, 4], device="cuda")[v + 2] + torch.where(v < 0, 8, 0)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), s


def sorted_slots(counts, B, k, seed):
    """order and offsets of R = sum(counts) sorted slots, slots drawn at random from B*k."""
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    order = torch.randperm(B * k, generator=gen(seed), device="cuda")[: int(off[-1])].to(torch.int32)
    return order, off


def expert_rows(off, R):
    at = torch.arange(R, device="cuda")
    return torch.searchsorted(off[1:].long(), at, right=True)


def products64(a, off, w):
    """float64 products of sorted rows and the sums of their absolute terms."""
    y = torch.full((a.shape[0], w.shape[1]), float("nan"), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    ends = off.tolist()
    for e in range(len(ends) - 1):
        rows = slice(ends[e], ends[e + 1])
        y[rows] = a[rows] @ w[e].T
        mag[rows] = a[rows].abs() @ w[e].abs().T
    return y, mag


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


# ---------------------------------------------------------------------------- norm

@pytest.mark.parametrize("B,H", [(1, 1), (1, 2048), (3, 31), (5, 256), (2, 1111), (7, 4096), (2, 4104), (3, 7168),
                                 (2, 8192), (1, 8200), (2, 16416), (1, 32768), (1, 32767), (2500, 96), (2049, 2048)])
@pytest.mark.parametrize("x_dtype,r_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                             (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16),
                                             (torch.bfloat16, None), (torch.float32, None)])
def test_norm(B, H, x_dtype, r_dtype):
    g = gen(B * 131 + H)
    x = (torch.randn(B, H, generator=g, device="cuda") * 2).to(x_dtype)
    r = None if r_dtype is None else (torch.randn(B, H, generator=g, device="cuda") * 3).to(r_dtype)
    for g_dtype in (torch.bfloat16, torch.float32):
        gain = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(g_dtype)
        quant = H % 32 == 0
        out, res, q, s = md.moe_norm(x, gain, residual=r, eps=1e-5, out_dtype=torch.float32, quantize=quant)
        v = x.double() if r is None else x.double() + r.double()
        y = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * gain.double()
        # the sum s, its square, the row's sum (halved by the root), root, two products
        tol = (H / 2 + 10) * U
        assert ((out.double() - y).abs() <= tol * y.abs() + 1e-30).all(), (g_dtype, float((out - y).abs().max()))
        if r is None:
            assert res is None
        else:
            assert torch.equal(bits(res), bits((x.float() + r.float()).to(r_dtype)))
        out16, _, q2, _ = md.moe_norm(x, gain, residual=r, eps=1e-5, quantize=quant)
        assert torch.equal(bits(out16), bits(out.to(torch.bfloat16)))
        if quant:
            assert torch.equal(q, q2)
            rq, rs = quantize(out)
            assert torch.equal(s, rs) and torch.equal(q, rq)
        else:
            assert q is None and s is None


def test_norm_in_place_and_without_plain_output():
    g = gen(5)
    x = torch.randn(9, 512, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(9, 512, generator=g, device="cuda").to(torch.bfloat16)
    gain = torch.ones(512, device="cuda")
    out, res, q, s = md.moe_norm(x, gain, residual=r, quantize=True)
    x2, r2 = x.clone(), r.clone()
    o2, res2, _, _ = md.moe_norm(x2, gain, residual=r2, residual_out=r2, out=x2)
    assert o2 is x2 and res2 is r2 and torch.equal(bits(x2), bits(out)) and torch.equal(bits(r2), bits(res))
    o3, _, q3, s3 = md.moe_norm(x, gain, residual=r, out_dtype=None, quantize=True)
    assert o3 is None and torch.equal(q, q3) and torch.equal(s, s3)


def test_norm_special_values():
    x = torch.randn(6, 96, generator=gen(6), device="cuda")
    x[0] = 0.0                                    # eps alone under the root
    x[1, 3] = float("nan")
    x[2, 40] = float("inf")
    x[3] *= 1e-38                                 # squares underflow
    x[4, :32] = 0.0                               # an all-zero block
    x[5, 70] = 3e19                               # the square overflows: 1 / inf
    gain = torch.ones(96, device="cuda")
    out, _, q, s = md.moe_norm(x, gain, out_dtype=torch.float32, quantize=True)
    assert torch.equal(out[0], torch.zeros(96, device="cuda")) and (s[0] == 0).all() and (q[0] == 0).all()
    assert out[1].isnan().all() and (s[1] == 255).all()
    assert out[2, 40].isnan() and (out[2, :32] == 0).all()
    assert list(s[2].cpu()) == [0, 255, 0]
    np.testing.assert_allclose(out[3].cpu(), x[3].double().cpu() * 1e3, rtol=1e-6)
    assert s[4, 0] == 0 and (q[4, :32] & 127 == 0).all() and (s[4, 1:] > 0).all()
    assert (out[5] == 0).all()
    rq, rs = quantize(out)
    assert torch.equal(s, rs) and torch.equal(q, rq)


# ---------------------------------------------------------------------------- group

@pytest.mark.parametrize("B,k,E", [(1, 1, 1), (1, 8, 128), (64, 8, 256), (3, 5, 67), (128, 8, 9), (129, 8, 9), (1000, 8, 128),
                                   (1024, 8, 2048), (1025, 8, 2048), (500, 8, 1700), (4097, 3, 31), (16384, 8, 128), (33000, 8, 64),
                                   (262144, 1, 3), (262145, 1, 1000), (7, 64, 64)])
@pytest.mark.parametrize("bad", [False, True])
def test_group(B, k, E, bad):
    ids = torch.randint(-2 if bad else 0, E + (3 if bad else 0), (B, k), generator=gen(B + k + E), device="cuda",
                        dtype=torch.int32)
    if bad and B > 2:
        ids[1, 0], ids[2, 0] = 2 ** 31 - 1, -2 ** 31
    order, position, offsets = md.moe_group(ids, E)
    flat = ids.reshape(-1).cpu().numpy()
    ok = np.flatnonzero((flat >= 0) & (flat < E))
    ref = ok[np.argsort(flat[ok], kind="stable")]
    pos = np.full(flat.size, -1)
    pos[ref] = np.arange(ref.size)
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))]))
    assert np.array_equal(position.cpu().numpy().reshape(-1), pos)
    assert np.array_equal(order.cpu().numpy(), np.concatenate([ref, np.full(flat.size - ref.size, -1)]))


def test_group_skewed_and_empty():
    ids = torch.full((5000, 4), 6, dtype=torch.int32, device="cuda")      # one expert with everything
    order, position, offsets = md.moe_group(ids, 8)
    at = torch.arange(20000, device="cuda", dtype=torch.int32)
    assert torch.equal(order, at) and torch.equal(position.reshape(-1), at)
    assert offsets.tolist() == [0] * 7 + [20000] * 2
    order, position, offsets = md.moe_group(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 8)
    assert order.numel() == 0 and position.shape == (0, 4) and offsets.tolist() == [0] * 9


# ---------------------------------------------------------------------------- products

# rows per expert: empty experts, single rows, whole and part tiles, one expert with everything
COUNTS = {"few": [0, 1, 2, 0, 17, 5], "mid": [33, 0, 64, 65, 1, 130], "one": [0, 0, 300], "single": [1],
          "large": [700, 0, 257, 256, 3, 128, 1025], "even": [64] * 40, "ones": [1] * 10 + [0] * 3, "threes": [3] * 40,
          "some": [20, 33, 7, 18, 22], "forty": [40, 1, 79]}


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("act", ["bf16", "mxfp8"])
@pytest.mark.parametrize("K,N", [(32, 32), (96, 64), (128, 160), (256, 256), (288, 96), (640, 128), (768, 512),
                                 (1024, 288), (1120, 64)])
def test_matmul_exact(counts, wformat, act, K, N):
    counts = COUNTS[counts]
    E, R = len(counts), sum(counts)
    g = gen(K * 7 + N + R)
    n_a = R + 3
    if act == "mxfp8":
        a, a_s = whole_mx(g, (n_a, K), "mxfp8")
        av = decode(a, a_s)
    else:
        a, a_s = (torch.randint(-8, 9, (n_a, K), generator=g, device="cuda") / 2).to(torch.bfloat16), None
        av = a.double()
    w_q, w_s = whole_mx(g, (E, N, K), wformat)
    order, off = sorted_slots(counts, n_a, 2, R)
    wv = decode(w_q, w_s, wformat)
    tail = 5
    long_order = torch.cat([order, torch.full((tail,), -1, dtype=torch.int32, device="cuda")])
    ref, mag = products64(av[order.long() // 2], off, wv)
    assert mag.max() < 2 ** 21                    # in steps of at least 1/2: exact in float32
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((R + tail, N), 7.0, dtype=dt, device="cuda")
        md.moe_grouped_matmul(a, off, w_q, w_s, order=long_order, k=2, a_s=a_s, out=out, wformat=wformat)
        assert (out[R:] == 7.0).all()
        assert torch.equal(out[:R], ref.float().to(dt)), (dt, float((out[:R].double() - ref).abs().max()))
    # rows in place: no order
    if R:
        direct = md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s, out_dtype=torch.float32, wformat=wformat)
        assert torch.equal(direct[:R], products64(av[:R], off, wv)[0].float())


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("act", ["bf16", "mxfp8"])
@pytest.mark.parametrize("K,N", [(32, 32), (96, 64), (256, 160), (768, 288)])
def test_gate_up(counts, wformat, act, K, N):
    """Exact gates and ups, so only the SwiGLU rounds: the exponential's argument by 2^-24 * |gate| * 1.45
    (relative error of the exponential), and exponential, reciprocal and three products by a few steps."""
    counts = COUNTS[counts]
    E, R = len(counts), sum(counts)
    g = gen(K * 11 + N + R)
    n_a = R + 3
    if act == "mxfp8":
        a, _ = whole_mx(g, (n_a, K), "mxfp8")
        a_s = torch.randint(121, 123, (n_a, K // 32), generator=g, device="cuda").to(torch.uint8)
        av = decode(a, a_s)
    else:
        a, a_s = (torch.randint(-8, 9, (n_a, K), generator=g, device="cuda") / 128).to(torch.bfloat16), None
        av = a.double()
    wg, wu = whole_mx(g, (E, N, K), wformat), whole_mx(g, (E, N, K), wformat)
    order, off = sorted_slots(counts, n_a, 2, R)
    gate, _ = products64(av[order.long() // 2], off, decode(*wg, wformat))
    up, _ = products64(av[order.long() // 2], off, decode(*wu, wformat))
    ref = gate * torch.sigmoid(gate) * up
    tol = (1.5 * gate.abs() + 16) * 2 * U
    call = lambda **kw: md.moe_grouped_gate_up(a, off, *wg, *wu, order=order, k=2, a_s=a_s, wformat=wformat, **kw)  # noqa: E731
    out = call(out_dtype=torch.float32)
    bad = (out.double() - ref).abs() > tol * ref.abs() + 1e-30
    assert not bad.any(), (int(bad.sum()), float((out.double() - ref).abs().max()))
    assert torch.equal(bits(call()), bits(out.to(torch.bfloat16)))
    q, s = call(quantize=True)
    rq, rs = quantize(out)
    assert torch.equal(s, rs) and torch.equal(q, rq)


@pytest.mark.parametrize("counts", ["few", "mid", "large"])
@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("act", ["bf16", "mxfp8"])
@pytest.mark.parametrize("K,N", [(2048, 96), (1056, 512)])
def test_matmul_rounding(counts, wformat, act, K, N):
    """Quantized normal values: float32 out within the bound of a float32 sum."""
    counts = COUNTS[counts]
    E, R = len(counts), sum(counts)
    g = gen(K + N + R)
    if act == "mxfp8":
        a, a_s = random_mx(g, (R, K), "mxfp8")
        av = decode(a, a_s)
    else:
        a, a_s = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16), None
        av = a.double()
    w_q, w_s = random_mx(g, (E, N, K), wformat, 0.02)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    ref, mag = products64(av, off, decode(w_q, w_s, wformat))
    out = md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s, out_dtype=torch.float32, wformat=wformat)
    err = (out.double() - ref).abs()
    assert (err <= 2 * K * U * mag).all(), float((err / mag).max() / U)
    rel = float(err.norm() / ref.norm())
    print(f"matmul {act} x {wformat} K={K}: relative 2-norm error {rel:.2e}", flush=True)
    # K roundings of independent sign: sqrt(K) * 2^-23 of the terms' 2-norm, which is below the magnitude's
    assert err.norm() <= 2 * K ** 0.5 * U * mag.norm()


def test_product_scales_of_every_size_and_nan():
    """MXFP8 rows and weights whose scales lie far apart, NaN scales and NaN codes."""
    K, N = 128, 32
    a = torch.full((4, K), 0x38, dtype=torch.uint8, device="cuda")                     # 1.0
    a_s = torch.full((4, K // 32), 127, dtype=torch.uint8, device="cuda")
    w_q = torch.full((1, N, K), 0x38, dtype=torch.uint8, device="cuda")
    w_s = torch.full((1, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    a_s[0] = 20
    w_s[0, 0] = 234                                # 2^-107 * 2^107
    a_s[1, 2] = 255
    w_s[0, 5, 1] = 255
    w_q[0, 6, 9] = 0x7F
    a[2, 100] = 0xFF
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    out = md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s, out_dtype=torch.float32)
    ref = decode(a, a_s) @ decode(w_q, w_s)[0].T
    assert torch.equal(out.isnan(), ref.isnan())
    assert torch.equal(out[~ref.isnan()], ref[~ref.isnan()].float())
    assert out[0, 0] == 128.0


def test_product_bad_order_makes_nan_rows():
    g = gen(3)
    K, N = 64, 64
    for counts in ([5, 0, 9], [300, 2, 500]):
        R = sum(counts)
        a = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16)
        w = random_mx(g, (3, N, K), "mxfp8")
        off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
        order = torch.arange(R, dtype=torch.int32, device="cuda")
        good = md.moe_grouped_matmul(a, off, *w, order=order)
        bad = torch.tensor([1, 4, R - 1], device="cuda")
        order[bad] = torch.tensor([-1, R, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        out = md.moe_grouped_matmul(a, off, *w, order=order)
        assert out[bad].isnan().all()
        keep = torch.ones(R, dtype=torch.bool, device="cuda")
        keep[bad] = False
        assert torch.equal(bits(out[keep]), bits(good[keep]))
        q, s = md.moe_grouped_gate_up(a, off, *w, *w, order=order, quantize=True)
        assert (s[bad] == 255).all() and (s[keep] != 255).all()


@pytest.mark.parametrize("K", [256, 480, 512, 640, 896])
def test_product_scales_at_dword_addresses(K):
    """Scale tensors are bytes at any multiple of four."""
    g = gen(8)
    counts = [20, 140]
    N, R = 96, 160
    a, a_s = whole_mx(g, (R, K), "mxfp8")
    w_q, w_s = whole_mx(g, (2, N, K), "mxfp8")
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    ref = md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s, out_dtype=torch.float32)
    assert torch.equal(ref, products64(decode(a, a_s), off, decode(w_q, w_s))[0].float())

    def moved(t, shift):
        room = torch.empty(t.numel() + shift, dtype=torch.uint8, device="cuda")
        room[shift:] = t.reshape(-1)
        return room[shift:].view(t.shape)

    for shift in (4, 8, 12):
        out = md.moe_grouped_matmul(a, off, w_q, moved(w_s, shift), a_s=moved(a_s, shift), out_dtype=torch.float32)
        assert torch.equal(out, ref), shift
    for bad in ({"w_s": moved(w_s, 2), "a_s": a_s}, {"w_s": w_s, "a_s": moved(a_s, 1)}):
        with pytest.raises(md.MoedError) as e:
            md.moe_grouped_matmul(a, off, w_q, **bad)
        assert e.value.status == md.MOED_ERR_ALIGN


@pytest.mark.parametrize("E", [1537, 2048])
def test_product_many_experts(E):
    """Average row counts of the largest tile, with more experts than its tile list has room for."""
    K, N = 128, 32
    g = gen(E)
    counts = np.random.default_rng(E).integers(60, 160, E)
    R = int(counts.sum())
    a, a_s = whole_mx(g, (R, K), "mxfp8")
    w_q, w_s = whole_mx(g, (E, N, K), "mxfp4")
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    wv, av = decode(w_q, w_s, "mxfp4"), decode(a, a_s)
    out = md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s, wformat="mxfp4")
    e = expert_rows(off, R)
    for some in torch.arange(R, device="cuda").split(20000):
        ref = (wv[e[some]] @ av[some][..., None]).squeeze(-1)
        assert torch.equal(out[some], ref.float().to(torch.bfloat16))


def test_product_past_32_bits():
    """More than 2^32 bytes of outputs, and of rows in place."""
    K, N, R = 128, 32736, 70001
    g = gen(77)
    a, a_s = whole_mx(g, (R, K), "mxfp8")
    w_q, w_s = whole_mx(g, (2, N, K), "mxfp8")
    off = torch.tensor([0, 5, R], dtype=torch.int32, device="cuda")
    out = md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s)
    assert out.numel() > 2 ** 31
    wv = decode(w_q, w_s)
    for r in (0, 4, 5, 33333, 65599, 65600, R - 1):
        assert torch.equal(out[r], (wv[int(r >= 5)] @ decode(a[r:r + 1], a_s[r:r + 1])[0]).float().to(torch.bfloat16)), r
    del out
    rows = torch.empty((70000, 32768), dtype=torch.bfloat16, device="cuda")
    rows[-300:] = torch.randint(-4, 5, (300, 32768), generator=g, device="cuda").to(torch.bfloat16)
    rows[:-300] = 0
    w_q, w_s = whole_mx(g, (1, 32, 32768), "mxfp4")
    out = md.moe_grouped_matmul(rows, torch.tensor([0, 70000], dtype=torch.int32, device="cuda"), w_q, w_s,
                                out_dtype=torch.float32, wformat="mxfp4")
    ref = rows[-300:].double() @ decode(w_q, w_s, "mxfp4")[0].T
    assert torch.equal(out[-300:], ref.float()) and (out[:-300] == 0).all()
    # gathered rows between 2 and 4 GiB: 32-bit offsets without a sign
    last = rows[-65535:]
    order = torch.tensor([65244, 2, 65534], dtype=torch.int32, device="cuda")
    out = md.moe_grouped_matmul(last, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), w_q, w_s, order=order,
                                out_dtype=torch.float32, wformat="mxfp4")
    assert torch.equal(out, (last[order.long()].double() @ decode(w_q, w_s, "mxfp4")[0].T).float())
    with pytest.raises(md.MoedError):            # gathered rows of 4 GiB and more are refused
        md.moe_grouped_matmul(rows, torch.tensor([0, 4], dtype=torch.int32, device="cuda"), w_q, w_s,
                              order=torch.arange(4, dtype=torch.int32, device="cuda"), wformat="mxfp4")


def test_product_offsets_that_make_no_sense():
    """Decreasing, negative and too large offsets: wrong rows, but the call ends and other rows stay as they were."""
    g = gen(12)
    K, N, R = 128, 64, 500
    a = torch.ones(R, K, dtype=torch.bfloat16, device="cuda")
    w_q, w_s = whole_mx(g, (4, N, K), "mxfp8")
    for off in ([0, 300, 100, 400, 450], [-5, 10, 20, 2 ** 31 - 1, 7], [500, 500, 500, 500, 500], [2 ** 31 - 1] * 5, [-1] * 5):
        out = torch.full((R + 2, N), 9.0, dtype=torch.float32, device="cuda")
        md.moe_grouped_matmul(a, torch.tensor(off, dtype=torch.int32, device="cuda"), w_q, w_s, out=out[:R])
        torch.cuda.synchronize()
        assert (out[R:] == 9.0).all()


# ---------------------------------------------------------------------------- combine

@pytest.mark.parametrize("B,k,H", [(1, 8, 2048), (3, 1, 7), (5, 64, 33), (300, 8, 4096), (17, 9, 2056), (2, 3, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine(B, k, H, dtype):
    g = gen(B + k + H)
    y = torch.randn(B * k, H, generator=g, device="cuda").to(dtype)
    pos = torch.randperm(B * k, generator=g, device="cuda").to(torch.int32).reshape(B, k)
    w = torch.rand(B, k, generator=g, device="cuda")
    terms = y.double()[pos.long()] * w.double()[..., None]
    out = md.moe_combine(y, pos, w, out_dtype=torch.float32)
    assert ((out.double() - terms.sum(1)).abs() <= (k + 1) * U * terms.abs().sum(1)).all()
    assert torch.equal(bits(md.moe_combine(y, pos, w)), bits(out.to(torch.bfloat16)))


def test_norm_and_combine_past_32_bits():
    B, H = 140000, 16384
    x = torch.empty((B, H), dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    x[-1] = torch.randn(H, generator=gen(1), device="cuda").to(torch.bfloat16)
    gain = torch.ones(H, device="cuda")
    out, _, q, s = md.moe_norm(x, gain, quantize=True)
    for b in (0, 131071, 131072, B - 1):
        one, _, q1, s1 = md.moe_norm(x[b:b + 1].clone(), gain, quantize=True)
        assert torch.equal(bits(out[b]), bits(one[0])) and torch.equal(q[b], q1[0]) and torch.equal(s[b], s1[0])
    pos = torch.tensor([[0, B - 1], [131072, 131071]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 2.0], [0.5, 0.25]], device="cuda")
    got = md.moe_combine(x, pos, w, out_dtype=torch.float32)
    assert torch.equal(got[0], x[0].float() + 2 * x[-1].float()) and (got[1] == 0.75).all()


def test_combine_bad_positions():
    y = torch.ones(6, 40, device="cuda")
    pos = torch.tensor([[0, 1], [2, -1], [6, 3], [2 ** 31 - 1, 4], [5, 5]], dtype=torch.int32, device="cuda")
    w = torch.ones(5, 2, device="cuda")
    out = md.moe_combine(y, pos, w, out_dtype=torch.float32)
    assert out[1:4].isnan().all() and (out[0] == 2).all() and (out[4] == 2).all()


# ---------------------------------------------------------------------------- the run of them

def layer_inputs(B, E, k, H, I, wformat, seed):
    g = gen(seed)
    x = torch.randn(B, H, generator=g, device="cuda")
    logits = torch.randn(B, E, generator=g, device="cuda")
    mats = []
    for N, K in ((I, H), (I, H), (H, I)):
        mats += list(random_mx(g, (E, N, K), wformat, 0.05))
    return x, logits, mats


@pytest.mark.parametrize("B,E,k,H,I", [(1, 8, 2, 256, 128), (7, 16, 4, 288, 96), (100, 16, 4, 256, 160),
                                       (1500, 8, 2, 512, 256), (3, 4, 4, 64, 32)])
@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("quantized", [False, True])
def test_block(B, E, k, H, I, wformat, quantized):
    """norm -> route -> prefill, against float64 with the intermediate rounded as the call rounds it.

    An intermediate value is off by at most half a step of its type (2^-8 in bfloat16, 2^-4 in E4M3 or half the
    smallest step of its block), and so is every product of it; the down rows and the output add 2^-8 each in
    bfloat16, sums 2^-23 per term."""
    x, logits, mats = layer_inputs(B, E, k, H, I, wformat, B + H)
    gain = torch.ones(H, device="cuda")
    r = torch.randn(B, H, generator=gen(9), device="cuda").to(torch.bfloat16)
    h, res, hq, hs = md.moe_norm(x.to(torch.bfloat16), gain, residual=r, quantize=quantized)
    ids, w = md.moe_route(logits, k)
    ids2 = ids.clone()
    if B > 4:
        ids2[3, 1] = ids2[3, 0]                   # the same expert twice
        ids2[4, 0] = -1
    for out_dtype in (torch.float32, torch.bfloat16):
        if quantized:
            out = md.moe_prefill(hq, ids2, w, *mats, x_s=hs, out_dtype=out_dtype, wformat=wformat)
            hv = decode(hq, hs)
        else:
            out = md.moe_prefill(h, ids2, w, *mats, out_dtype=out_dtype, wformat=wformat)
            hv = h.double()
        wg, wu, wd = (decode(*mats[i:i + 2], wformat) for i in (0, 2, 4))
        for b in sorted({0, B // 2, B - 1, min(B - 1, 3)}):
            ref = torch.zeros(H, dtype=torch.float64, device="cuda")
            tol = torch.zeros_like(ref)
            for j in range(k):
                e = int(ids2[b, j])
                if not 0 <= e < E:
                    ref += float("nan")
                    continue
                gate, up = wg[e] @ hv[b], wu[e] @ hv[b]
                a = gate * torch.sigmoid(gate) * up
                if quantized:
                    top = a.unflatten(0, (-1, 32)).abs().amax(-1, keepdim=True)
                    step = torch.maximum(a.unflatten(0, (-1, 32)).abs() * 2.0 ** -4, top * 2.0 ** -17)
                    # between 448 and 512 of a block's scale codes saturate: off by at most an eighth
                    step = torch.where(a.unflatten(0, (-1, 32)).abs() >= top / 512 * 448 * 0.99, top / 8, step).flatten()
                else:
                    step = a.abs() * BF16
                mag_g, mag_u = wg[e].abs() @ hv[b].abs(), wu[e].abs() @ hv[b].abs()
                step = step + 2 * H * U * (mag_g * up.abs() * 1.1 + mag_u * gate.abs()) + 32 * U * a.abs()
                y = wd[e] @ a
                d = wd[e].abs() @ (step + 2 * I * U * a.abs())
                if out_dtype == torch.bfloat16:
                    d = d + (y.abs() + d) * BF16
                ref += w[b, j].double() * y
                tol += w[b, j].double() * (d + (k + 1) * U * y.abs())
            if out_dtype == torch.bfloat16:
                tol = tol + (ref.abs() + tol) * BF16
            got = out[b].double()
            if ref.isnan().any():
                assert got.isnan().all()
            else:
                assert ((got - ref).abs() <= tol).all(), (b, float(((got - ref).abs() / tol).max()))
        if B > 4:
            assert out[4].isnan().all()


def test_prefill_agrees_with_decode():
    """bfloat16 rows: the same layer as moe_decode with a bfloat16 intermediate; their float32 sums differ in order
    only, so an intermediate value can differ by one bfloat16 step where a sum lies next to a border."""
    x, logits, mats = layer_inputs(40, 16, 4, 512, 256, "mxfp8", 21)
    x = x.to(torch.bfloat16)
    ids, w = md.moe_route(logits, 4)
    ref = md.moe_decode(x, ids, w, *mats, out_dtype=torch.float32, inter_dtype=torch.bfloat16)
    out = md.moe_prefill(x, ids, w, *mats, out_dtype=torch.float32)
    rel = float((out.double() - ref.double()).norm() / ref.double().norm())
    assert rel <= 2 * BF16, rel


def test_prefill_check_mode(monkeypatch):
    x, logits, mats = layer_inputs(6, 8, 2, 64, 32, "mxfp8", 4)
    x = x.to(torch.bfloat16)
    ids, w = md.moe_route(logits, 2)
    monkeypatch.setenv("MOED_CHECK", "1")
    md.moe_prefill(x, ids, w, *mats)
    bad = ids.clone()
    bad[2, 1] = 8
    with pytest.raises(md.MoedError) as e:
        md.moe_prefill(x, bad, w, *mats)
    assert e.value.status == md.MOED_ERR_SHAPE
    mats[1][int(ids[0, 0]), 3, 1] = 250           # outside the range that the conversion holds exactly
    with pytest.raises(md.MoedError) as e:
        md.moe_prefill(x, ids, w, *mats)
    assert e.value.status == md.MOED_ERR_SCALE
    # MXFP8 rows take any scale in the gate and up matrices; in the down matrix only where float32 is not asked for
    hq, hs = quantize(x.float())
    md.moe_prefill(hq, ids, w, *mats, x_s=hs, out_dtype=torch.float32)
    mats[5][int(ids[0, 0]), 3, 0] = 250
    md.moe_prefill(hq, ids, w, *mats, x_s=hs)
    with pytest.raises(md.MoedError):
        md.moe_prefill(hq, ids, w, *mats, x_s=hs, out_dtype=torch.float32)


def run_block(x, r, gain, logits, mats, k, ws=None, stream=None):
    h, res, hq, hs = md.moe_norm(x, gain, residual=r, quantize=True, stream=stream)
    ids, w = md.moe_route(logits, k, stream=stream)
    return h, res, hq, hs, ids, w, md.moe_prefill(hq, ids, w, *mats, x_s=hs, workspace=ws, stream=stream)


def test_block_captured_and_replayed():
    x, logits, mats = layer_inputs(600, 16, 4, 256, 128, "mxfp8", 31)
    x = x.to(torch.bfloat16)
    r = torch.randn(600, 256, generator=gen(2), device="cuda").to(torch.bfloat16)
    gain = torch.ones(256, device="cuda")
    run_block(x, r, gain, logits, mats, 4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_block(x, r, gain, logits, mats, 4)
    for i in range(4):
        x.copy_(torch.randn(600, 256, generator=gen(40 + i), device="cuda"))
        logits.copy_(torch.randn(600, 16, generator=gen(50 + i), device="cuda"))
        want = run_block(x, r, gain, logits, mats, 4)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(bits(a), bits(b)), i


def test_block_on_two_streams_at_once():
    shapes = [(300, 16, 4, 256, 128), (40, 16, 4, 256, 128)]
    sets = [(layer_inputs(*s, "mxfp8", 60 + i), s) for i, s in enumerate(shapes)]
    gain = torch.ones(256, device="cuda")
    rs = [torch.randn(s[0], 256, generator=gen(70), device="cuda").to(torch.bfloat16) for s in shapes]
    want = [run_block(i[0].to(torch.bfloat16), r, gain, i[1], i[2], 4) for (i, s), r in zip(sets, rs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for st, (i, s), r in zip(streams, sets, rs):
            st.wait_stream(torch.cuda.current_stream())
            xb = i[0].to(torch.bfloat16)
            st.wait_stream(torch.cuda.current_stream())
            got.append((xb, run_block(xb, r, gain, i[1], i[2], 4, stream=st)))
        torch.cuda.synchronize()
        for (_, a), b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(bits(u), bits(v))


def test_raw_stream_handle():
    """A stream given as its handle, with everything made inside the calls."""
    x, logits, mats = layer_inputs(30, 16, 4, 288, 96, "mxfp8", 91)
    x = x.to(torch.bfloat16)
    gain, r = torch.ones(288, device="cuda"), torch.zeros(30, 288, dtype=torch.bfloat16, device="cuda")
    want = run_block(x, r, gain, logits, mats, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run_block(x, r, gain, logits, mats, 4, stream=side.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))


def test_results_repeat():
    x, logits, mats = layer_inputs(900, 16, 4, 512, 256, "mxfp4", 81)
    x = x.to(torch.bfloat16)
    ids, w = md.moe_route(logits, 4)
    ref = md.moe_prefill(x, ids, w, *mats, wformat="mxfp4")
    for _ in range(3):
        assert torch.equal(bits(md.moe_prefill(x, ids, w, *mats, wformat="mxfp4")), bits(ref))


def test_empty_calls():
    e = torch.empty
    dev = {"device": "cuda"}
    out, res, q, s = md.moe_norm(e(0, 64, dtype=torch.bfloat16, **dev), e(64, **dev), quantize=True)
    assert out.shape == (0, 64) and q.shape == (0, 64) and s.shape == (0, 2) and res is None
    w_q, w_s = e(2, 32, 64, dtype=torch.uint8, **dev), e(2, 32, 2, dtype=torch.uint8, **dev)
    off = torch.zeros(3, dtype=torch.int32, **dev)
    assert md.moe_grouped_matmul(e(0, 64, dtype=torch.bfloat16, **dev), off, w_q, w_s).shape == (0, 32)
    assert md.moe_combine(e(0, 64, **dev), e(0, 2, dtype=torch.int32, **dev), e(0, 2, **dev)).shape == (0, 64)
    d_q, d_s = e(2, 64, 32, dtype=torch.uint8, **dev), e(2, 64, 1, dtype=torch.uint8, **dev)
    assert md.moe_prefill(e(0, 64, dtype=torch.bfloat16, **dev), e(0, 2, dtype=torch.int32, **dev), e(0, 2, **dev),
                          w_q, w_s, w_q, w_s, d_q, d_s).shape == (0, 64)
    # experts that exist but got no row: the outputs stay
    a = torch.ones(4, 64, dtype=torch.bfloat16, **dev)
    out = torch.full((4, 32), 3.0, **dev)
    md.moe_grouped_matmul(a, off, w_q, w_s, out=out)
    assert (out == 3.0).all()


def test_binding_refusals():
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    gain = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        md.moe_norm(x.t().contiguous().t(), gain)                 # strides
    with pytest.raises(ValueError):
        md.moe_norm(x.cpu(), gain)
    with pytest.raises(ValueError):
        md.moe_norm(x, gain[:32])
    with pytest.raises(TypeError):
        md.moe_norm(x.half(), gain)
    with pytest.raises(ValueError):
        md.moe_norm(torch.ones(4, 48, device="cuda"), torch.ones(48, device="cuda"), quantize=True)
    with pytest.raises(TypeError):
        md.moe_norm(x, gain, residual=x, residual_out=x.float())
    with pytest.raises(TypeError):
        md.moe_group(torch.zeros(2, 2, dtype=torch.int64, device="cuda"), 4)
    with pytest.raises(md.MoedError):
        md.moe_group(torch.zeros(2, 2, dtype=torch.int32, device="cuda"), 4096)
    w_q, w_s = torch.zeros(2, 32, 64, dtype=torch.uint8, device="cuda"), torch.zeros(2, 32, 2, dtype=torch.uint8, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        md.moe_grouped_matmul(x, off[:2], w_q, w_s)
    with pytest.raises(ValueError):
        md.moe_grouped_matmul(x, off, w_q, w_s, wformat="mxfp4")
    with pytest.raises(TypeError):
        md.moe_grouped_matmul(x, off, w_q, w_s, a_s=w_s[0])       # bfloat16 rows with scales
    with pytest.raises(ValueError):                               # scales of an output that is not MXFP8
        md.moe_grouped_gate_up(x, off, w_q, w_s, w_q, w_s, out_s=torch.zeros(4, 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(md.MoedError):
        md.moe_grouped_matmul(x, off, w_q, w_s, order=torch.zeros(4, dtype=torch.int32, device="cuda"), k=0)
    with pytest.raises(md.MoedError):
        room = torch.zeros(2 * 32 * 64 + 4, dtype=torch.uint8, device="cuda")
        md.moe_grouped_matmul(x, off, room[4:].view(2, 32, 64), w_s)


def test_norm_past_the_range():
    """Squares whose float32 sum is infinite: zeros, and the sum with the residual as it is."""
    x = torch.full((2, 64), 2.0 ** 70, device="cuda")
    x[1] = 1.0
    out, res, q, s = md.moe_norm(x, torch.ones(64, device="cuda"), residual=x, eps=0.0, out_dtype=torch.float32, quantize=True)
    assert (out[0] == 0).all() and (q[0] == 0).all() and (s[0] == 0).all()
    # row 1: one unit in the last place of the reciprocal root, one rounding of the product
    assert torch.equal(res, 2 * x) and ((out[1] - 1).abs() <= 2.0 ** -22).all()
