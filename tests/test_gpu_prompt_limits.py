"""GPU tests of the prompt-side operators at the ends of their ranges: the sums behind bfloat16 and MXFP8 outputs of
MXFP8 rows, block scales of every size, NaN, tiny rows, long lists and large tensors.

A float32 sum of K terms is off by at most 2^-23 a term of the sum of their magnitudes (test_gpu_prompt). What the
scaled matrix instructions (fast) drop measured 1.4e-5 to 1.5e-5 of the result in the 2-norm with normal values. It is
a sum of many small parts, so a single output is held to ten times that, of the 2-norm of its own terms, and a 2-norm
over thousands of outputs to twice that. Rounding keeps order, so an output whose unrounded value lies within d of the
exact y lies between the roundings of y - d and y + d."""
import numpy as np
import pytest
import torch

from output_centric_expert_amd import moedecode as md
from test_gpu_prompt import (COUNTS, U, decode, gen, gpu, layer_inputs, products64, quantize, random_mx,  # noqa: F401
                             whole_mx)

pytestmark = pytest.mark.gpu

DROPPED = 1.4e-5


def ones(shape, fmt):
    """Codes of 1.0."""
    K = shape[-1] if fmt == "mxfp8" else shape[-1] // 2
    return torch.full((*shape[:-1], K), 0x38 if fmt == "mxfp8" else 0x22, dtype=torch.uint8, device="cuda")


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------- sums of MXFP8 rows

def eights(K, R):
    """Rows with 256, -256 and six times 2^-6 in every eight values: sums that lose their small terms where an eight is
    aligned to its largest."""
    v = torch.full((R, K), 2.0 ** -6, device="cuda")
    v[:, 0::8], v[:, 3::8] = 256.0, -256.0
    return (v.to(torch.float8_e4m3fn).view(torch.uint8),
            torch.full((R, K // 32), 127, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("rows", [1, 5, 20, 40, 100, 300])
@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("K", [96, 512, 1152])
def test_rounded_outputs_are_of_whole_sums(rows, wformat, K):
    """Weights of 64: every product is a whole number and every sum below 2^24, exact in float32 in any order."""
    N = 96
    a, a_s = eights(K, rows)
    w_q = ones((1, N, K), wformat)
    w_s = torch.full((1, N, K // 32), 133, dtype=torch.uint8, device="cuda")
    off = offsets_of([rows])
    want = 6 * K // 8
    out = md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s, wformat=wformat)
    assert (out == want).all()                    # 72, 384 and 864 are bfloat16 values
    u_s = w_s - 3                                 # ups of an eighth
    kw = {"a_s": a_s, "wformat": wformat}
    y = md.moe_grouped_gate_up(a, off, w_q, w_s, w_q, u_s, out_dtype=torch.float32, **kw)
    assert (y == want * want / 8).all()           # SiLU of 72 and more is its argument
    assert torch.equal(md.moe_grouped_gate_up(a, off, w_q, w_s, w_q, u_s, **kw), y.to(torch.bfloat16))
    q, s = md.moe_grouped_gate_up(a, off, w_q, w_s, w_q, u_s, quantize=True, **kw)
    rq, rs = quantize(y)
    assert torch.equal(q, rq) and torch.equal(s, rs)


@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts", ["few", "mid", "large"])
def test_scales_outside_the_exact_range(wformat, counts):
    """Rows times 2^-123 in one block of 32 and 2^123 in another, weights the other way round: the same whole sums."""
    counts = COUNTS[counts]
    E, R, K, N = len(counts), sum(counts), 640, 96
    g = gen(R)
    a, a_s = whole_mx(g, (R, K), "mxfp8")
    w_q, w_s = whole_mx(g, (E, N, K), wformat)
    u_q, u_s = whole_mx(g, (E, N, K), wformat)
    off = offsets_of(counts)
    plain = md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s, wformat=wformat)
    q, s = md.moe_grouped_gate_up(a, off, w_q, w_s, u_q, u_s, a_s=a_s, quantize=True, wformat=wformat)
    for block, by in ((4, 123), (19, -123)):
        a_s[:, block] = (a_s[:, block].int() - by).to(torch.uint8)
        w_s[:, :, block] = (w_s[:, :, block].int() + by).to(torch.uint8)
        u_s[:, :, block] = (u_s[:, :, block].int() + by).to(torch.uint8)
    assert torch.equal(md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s, wformat=wformat), plain)
    q2, s2 = md.moe_grouped_gate_up(a, off, w_q, w_s, u_q, u_s, a_s=a_s, quantize=True, wformat=wformat)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("K", [256, 224])
def test_scales_outside_the_exact_range_change_their_tiles_only(wformat, K):
    """A block with such a scale makes its tile lose the small terms of its eights; other tiles keep theirs, and blocks
    of zeros may have any scale."""
    N, R = 256, 700
    a, a_s = eights(K, R)
    w_q = ones((2, N, K), wformat)
    w_s = torch.full((2, N, K // 32), 133, dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 350, R], dtype=torch.int32, device="cuda")
    call = lambda: md.moe_grouped_matmul(a, off, w_q, w_s, a_s=a_s, wformat=wformat)  # noqa: E731
    whole, block = 6 * K // 8, 24
    assert (call() == whole).all()
    a[690, 32:96] = 0
    a_s[690, 1], a_s[690, 2] = 0, 254
    w_q[1, 7, : w_q.shape[2] * 32 // K] = 0
    w_s[1, 7, 0] = 1
    want = torch.full((R, N), float(whole), device="cuda")
    want[690] -= 2 * block
    want[350:, 7] -= block
    assert torch.equal(call().float(), want)
    a_s[690, 5] = 3
    out = call().float()
    assert torch.equal(out[:350], want[:350])
    lost = (out[350:] == 0) | (out[350:] == want[350:])
    lost[340] = True
    assert lost.all()
    if wformat == "mxfp8":                        # the tile was computed with the scaled instructions
        assert (out[691, 8:] == 0).all()


# ---------------------------------------------------------------------------- every scale, NaN, error

SCALES = (0, 1, 2, 10, 54, 60, 64, 100, 126, 127, 128, 150, 190, 245, 253, 254, 255)


@pytest.mark.parametrize("K", [96, 128, 512, 1152])
@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("rows_each", [1, 40])
@pytest.mark.parametrize("fast", [False, True])
def test_product_takes_every_scale(K, wformat, rows_each, fast):
    """Every pair of a row's and a weight's scale code: K * 2^(s + t - 254), NaN where either is 255."""
    a_s = torch.tensor(SCALES, dtype=torch.uint8, device="cuda").repeat_interleave(rows_each)
    R, N = a_s.numel(), 32
    w_s = torch.full((N,), 127, dtype=torch.uint8, device="cuda")
    w_s[:len(SCALES)] = torch.tensor(SCALES, dtype=torch.uint8, device="cuda")
    out = md.moe_grouped_matmul(ones((R, K), "mxfp8"), offsets_of([R]), ones((1, N, K), wformat),
                                w_s[None, :, None].expand(1, N, K // 32).contiguous(),
                                a_s=a_s[:, None].expand(R, K // 32).contiguous(), wformat=wformat, fast=fast)
    two = K * torch.exp2(a_s.double()[:, None] + w_s.double() - 254)
    # the sum is K times a power of two: exact in float32 (54 + 64 gives subnormal values, which stay), and K = 96 .. 1152
    # in bfloat16 too, unless subnormal
    ref = two.float().to(torch.bfloat16)
    nan = (a_s == 255)[:, None] | (w_s == 255)
    assert torch.equal(out.isnan(), nan)
    assert torch.equal(out[~nan], ref[~nan])


@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("fast", [False, True])
def test_rounded_product_nan(wformat, fast):
    """One NaN code or scale makes the outputs that it enters NaN and leaves the others; in an MXFP8 output a block
    with a NaN has scale 255 and NaN codes."""
    g = gen(17)
    K, N, R = 640, 64, 70
    a, a_s = whole_mx(g, (R, K), "mxfp8")
    w = whole_mx(g, (1, N, K), wformat)
    u = whole_mx(g, (1, N, K), wformat)
    off = offsets_of([R])
    good = md.moe_grouped_matmul(a, off, *w, a_s=a_s, wformat=wformat, fast=fast)
    gq, gs = md.moe_grouped_gate_up(a, off, *w, *u, a_s=a_s, quantize=True, wformat=wformat, fast=fast)
    a_s[3, 7] = 255
    a[40, 600] = 0x7F
    a[69, 0] = 0xFF
    w[1][0, 5, 19] = 255
    rows, cols = [3, 40, 69], [5]
    if wformat == "mxfp8":
        w[0][0, 33, 130] = 0x7F
        cols.append(33)
    nan = torch.zeros(R, N, dtype=torch.bool, device="cuda")
    nan[rows] = True
    nan[:, cols] = True
    out = md.moe_grouped_matmul(a, off, *w, a_s=a_s, wformat=wformat, fast=fast)
    assert torch.equal(out.isnan(), nan) and torch.equal(out[~nan], good[~nan])
    q, s = md.moe_grouped_gate_up(a, off, *w, *u, a_s=a_s, quantize=True, wformat=wformat, fast=fast)
    blocks = nan.unflatten(1, (-1, 32)).any(2)
    assert torch.equal(s == 255, blocks)
    assert torch.equal(q == 0x7F, blocks.repeat_interleave(32, 1))
    assert torch.equal(s[~blocks], gs[~blocks])
    keep = ~blocks.repeat_interleave(32, 1)
    assert torch.equal(q[keep], gq[keep])


@pytest.mark.parametrize("K", [512, 2048, 7168])
@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("fast", [False, True])
def test_rounded_product_error(K, wformat, fast):
    """Float32 sums behind rounded outputs, and the stated 2-norm of what fast drops. Four digits of minus the product, met by rows that are 1 in one place,
    leave little but the error in the output, so that its bfloat16 rounding hides nothing."""
    g = gen(K)
    R, N = 32, 96

    def encode(v):
        if wformat == "mxfp8":
            return quantize(v)
        amax = v.unflatten(-1, (-1, 32)).abs().amax(-1)
        s = (torch.frexp(amax)[1] - 3 + 127).to(torch.uint8)
        t = torch.ldexp(v.unflatten(-1, (-1, 32)), (127 - s.int())[..., None]).flatten(-2)
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
        c = (t.abs()[..., None] - table).abs().argmin(-1) + torch.where(t < 0, 8, 0)
        return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8), s

    a, a_s = random_mx(g, (R, K), "mxfp8")
    w, w_s = random_mx(g, (N, K), wformat, 0.02)
    main = decode(a, a_s) @ decode(w, w_s, wformat).T
    rest, codes, scales = -main, [], []
    for _ in range(4):
        c, s = encode(rest.T.float().contiguous())
        rest = rest - decode(c, s, wformat).T
        codes.append(c)
        scales.append(s)
    places = torch.eye(32, device="cuda").repeat(1, 4)
    p, p_s = quantize(places)
    rows, row_s = torch.cat([a, p], 1), torch.cat([a_s, p_s], 1)
    wq, ws = torch.cat([w, *codes], 1)[None].contiguous(), torch.cat([w_s, *scales], 1)[None].contiguous()
    ref = decode(rows, row_s) @ decode(wq, ws, wformat)[0].T
    out = md.moe_grouped_matmul(rows, offsets_of([R]), wq, ws, a_s=row_s, wformat=wformat, fast=fast)
    err = float((out.double() - ref).norm() / main.norm())
    print(f"product {wformat} K={K} fast={fast}: {err:.2e} of the product's 2-norm", flush=True)
    # the remainder's own rounding, and K roundings or truncations of independent sign of partial sums that are no larger
    # than the product
    assert float(ref.norm() / main.norm()) < 1e-3
    tol = 2.0 ** -8 * float(ref.norm() / main.norm()) + 2 * (K + 128) ** 0.5 * U
    assert err <= tol + (2 * DROPPED if fast else 0)


@pytest.mark.parametrize("counts", ["few", "mid", "large", "some"])
@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("K,N", [(2048, 96), (768, 512), (1056, 160)])
@pytest.mark.parametrize("fast", [False, True])
def test_rounded_outputs_lie_next_to_the_exact_ones(counts, wformat, K, N, fast):
    counts = COUNTS[counts]
    E, R = len(counts), sum(counts)
    g = gen(K + N + R)
    a, a_s = random_mx(g, (R, K), "mxfp8")
    wg, wu = random_mx(g, (E, N, K), wformat, 0.02), random_mx(g, (E, N, K), wformat, 0.02)
    off = offsets_of(counts)
    av = decode(a, a_s)

    def product(w):
        v = decode(*w, wformat)
        y, mag = products64(av, off, v)
        sq, _ = products64(av * av, off, v * v)
        return y, (10 * DROPPED * sq.sqrt() if fast else 0) + 2 * K * U * mag

    gate, dg = product(wg)
    out = md.moe_grouped_matmul(a, off, *wg, a_s=a_s, wformat=wformat, fast=fast)
    lo, hi = (gate - dg).float().to(torch.bfloat16), (gate + dg).float().to(torch.bfloat16)
    assert ((out >= lo) & (out <= hi)).all()
    up, du = product(wu)
    silu = gate * torch.sigmoid(gate)
    y = silu * up
    # SiLU' is at most 1.1; the SwiGLU itself as in the tests of exact gates
    d = 1.1 * dg * (up.abs() + du) + silu.abs() * du + (1.5 * gate.abs() + 16) * 2 * U * y.abs()
    q, s = md.moe_grouped_gate_up(a, off, *wg, *wu, a_s=a_s, quantize=True, wformat=wformat, fast=fast)
    yb, db = y.unflatten(1, (-1, 32)), d.unflatten(1, (-1, 32))
    low = quantize((yb.abs() - db).clamp(min=0).float().flatten(1))[1]
    high = quantize((yb.abs() + db).float().flatten(1))[1]
    assert ((s >= low) & (s <= high)).all()
    two = torch.exp2(127 - s.double())[..., None]

    def code(v):
        return (v * two).clamp(-448, 448).float().to(torch.float8_e4m3fn).float().flatten(1)

    v = q.view(torch.float8_e4m3fn).float()
    assert ((v >= code(yb - db)) & (v <= code(yb + db))).all()
    moved = float((v != code(yb)).float().mean())
    print(f"gate_up {wformat} K={K} N={N} R={R} fast={fast}: {moved:.2e} of the codes take a neighbour", flush=True)


@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("fast", [False, True])
def test_rounded_results_repeat(wformat, fast):
    """Bits of an MXFP8 layer of many tiles, call after call and through another tile list."""
    g = gen(23)
    E, K, N, R = 24, 768, 512, 5000
    a, a_s = random_mx(g, (R, K), "mxfp8")
    wg, wu = random_mx(g, (E, N, K), wformat, 0.02), random_mx(g, (E, N, K), wformat, 0.02)
    cuts = torch.randint(0, R + 1, (E - 1,), generator=g, device="cuda").sort().values
    off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), R)]).to(torch.int32)
    first = md.moe_grouped_gate_up(a, off, *wg, *wu, a_s=a_s, quantize=True, wformat=wformat, fast=fast)
    down = md.moe_grouped_matmul(a, off, *wg, a_s=a_s, wformat=wformat, fast=fast)
    for _ in range(4):
        again = md.moe_grouped_gate_up(a, off, *wg, *wu, a_s=a_s, quantize=True, wformat=wformat, fast=fast)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert torch.equal(down, md.moe_grouped_matmul(a, off, *wg, a_s=a_s, wformat=wformat, fast=fast))


# ---------------------------------------------------------------------------- sizes

@pytest.mark.parametrize("act,K,R", [("bf16", 2880, 800_000), ("mxfp8", 1056, 4_100_000)])
def test_rows_in_place_past_4_gib_with_padded_scales(act, K, R):
    """Rows in place beyond 2^32 bytes whose K needs its scales copied to the workspace."""
    g = gen(K)
    N, some = 32, 500
    wq, ws = whole_mx(g, (2, N, K), "mxfp8")
    off = torch.tensor([0, R - some, R], dtype=torch.int32, device="cuda")
    if act == "bf16":
        a, a_s = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda"), None
        a[-some:] = torch.randint(-4, 5, (some, K), generator=g, device="cuda").to(torch.bfloat16)
        tail = a[-some:].double()
    else:
        a = torch.zeros((R, K), dtype=torch.uint8, device="cuda")
        a_s = torch.full((R, K // 32), 127, dtype=torch.uint8, device="cuda")
        a[-some:], a_s[-some:] = whole_mx(g, (some, K), "mxfp8")
        tail = decode(a[-some:], a_s[-some:])
    assert a.numel() * a.element_size() > 2 ** 32
    out = md.moe_grouped_matmul(a, off, wq, ws, a_s=a_s)
    assert torch.equal(out[-some:], (tail @ decode(wq, ws)[1].T).float().to(torch.bfloat16))
    assert (out[:-some] == 0).all()


# ---------------------------------------------------------------------------- norm of tiny rows

@pytest.mark.parametrize("B,H", [(3, 96), (2500, 96), (2, 31), (3, 2048), (2, 4104), (1, 8200), (1, 32768), (1, 32767)])
@pytest.mark.parametrize("x_dtype,r_dtype", [(torch.float32, torch.float32), (torch.bfloat16, None),
                                             (torch.bfloat16, torch.bfloat16)])
def test_norm_of_tiny_rows(B, H, x_dtype, r_dtype):
    """Rows whose squares leave float32's range below, with an eps that does not hide it."""
    g = gen(B + H)
    # below 2^-149 / 2^-133 a value is 0 already; 2^-39 and 2^-41 lie on both sides of where squares get small
    for size in (1e-44, 1e-38, 1e-25, 1e-21, 2.0 ** -41, 2.0 ** -39):
        x = (torch.randn(B, H, generator=g, device="cuda", dtype=torch.float64) * size).to(x_dtype)
        x[:, 0] = size                            # no row of zeros
        if H > 40:
            x[0, 5:9] = 0.0
        r = None if r_dtype is None else (torch.randn(B, H, generator=g, device="cuda", dtype=torch.float64) * size).to(r_dtype)
        gain = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
        s = (x.cpu().float() if r is None else x.cpu().float() + r.cpu().float()).cuda().double()
        quant = H % 32 == 0
        for eps in (0.0, 1e-42, 1e-30, 1e-25, 1e-20):
            out, res, q, sc = md.moe_norm(x, gain, residual=r, eps=eps, out_dtype=torch.float32, quantize=quant)
            e = float(torch.tensor(eps, dtype=torch.float32))
            root = torch.sqrt((s * s).mean(1, keepdim=True) + e)
            s_ok = (root > 0).expand_as(s)        # a row may have rounded, or cancelled, to zeros
            y = s / root * gain.double()
            # the row's sum of squares, root and products as for other rows; below 2^-126 values have absolute steps
            tol = (H / 2 + 10) * U * y.abs() + 2.0 ** -148
            assert ((out.double() - y).abs() <= tol)[s_ok].all(), (size, eps)
            if r is not None:
                assert torch.equal(res.double(), s.float().to(r_dtype).double())
            if quant:
                rq, rs = quantize(out)
                assert torch.equal(sc, rs) and torch.equal(q, rq)


def test_norm_of_a_row_of_zeros():
    """0 / sqrt(eps), and 0 / 0 without an eps."""
    x = torch.zeros(2, 64, device="cuda")
    x[1] = 1e-30
    gain = torch.ones(64, device="cuda")
    out, _, q, s = md.moe_norm(x, gain, eps=0.0, out_dtype=torch.float32, quantize=True)
    assert out[0].isnan().all() and (s[0] == 255).all() and ((out[1] - 1).abs() <= 2.0 ** -22).all()
    out, _, q, s = md.moe_norm(x, gain, eps=1e-45, out_dtype=torch.float32, quantize=True)
    assert (out[0] == 0).all() and (s[0] == 0).all() and (q[0] == 0).all()


# ---------------------------------------------------------------------------- padded scales

@pytest.mark.parametrize("offsets", [[0, 0, 3, 3, 3, 9, 9], [0, 7, 5, 9, 2, 2, 9], [4, -2, 1, 30, 2, 9, 9]])
def test_padded_scales_of_experts_with_rows_only(offsets):
    """Where scales are copied to the workspace, experts without rows are left out; offsets that make no sense still
    give every row that a tile computes its scales."""
    g = gen(11)
    E, K, N, R = 6, 96, 64, 9
    a = torch.randint(-4, 5, (R, K), generator=g, device="cuda").to(torch.bfloat16)
    w, u = whole_mx(g, (E, N, K), "mxfp8"), whole_mx(g, (E, N, K), "mxfp8")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    # what a tile list makes of them: clamped to the rows, and rising
    rising = np.maximum.accumulate(np.clip(offsets, 0, R))
    ws = torch.full((md.moe_grouped_workspace_bytes(E, K, N, R, matrices=2),), 0x5A, dtype=torch.uint8, device="cuda")
    md.moe_grouped_gate_up(a, off, *w, *u, workspace=ws)
    copied = (ws.view(2, E, N * 16) != 0x5A).any(2).cpu().numpy()
    rows = rising[1:] > rising[:-1]
    asked = np.array(offsets[1:]) > np.array(offsets[:-1])
    assert not (rows & ~asked).any()
    assert (copied == asked).all()
    ws = torch.full((md.moe_grouped_workspace_bytes(E, K, N, R),), 0x5A, dtype=torch.uint8, device="cuda")
    out = md.moe_grouped_matmul(a, off, *w, out_dtype=torch.float32, workspace=ws)
    wv = decode(*w)
    for e in range(E):
        some = slice(int(rising[e]), int(rising[e + 1]))
        assert torch.equal(out[some], (a[some].double() @ wv[e].T).float())


# ---------------------------------------------------------------------------- long lists of slots

@pytest.mark.parametrize("B,k,E", [(262144, 8, 5), (262145, 8, 5), (300000, 8, 1), (300000, 8, 300), (65537, 64, 63),
                                   (300001, 7, 64), (300001, 7, 65), (300000, 8, 1700), (2400000, 1, 2048)])
@pytest.mark.parametrize("bad", [False, True])
def test_group_of_many_slots(B, k, E, bad):
    ids = torch.randint(-2 if bad else 0, E + (3 if bad else 0), (B, k), generator=gen(B + k + E), device="cuda",
                        dtype=torch.int32)
    order, position, offsets = md.moe_group(ids, E)
    flat = ids.reshape(-1).cpu().numpy()
    ok = np.flatnonzero((flat >= 0) & (flat < E))
    ref = ok[np.argsort(flat[ok], kind="stable")]
    pos = np.full(flat.size, -1)
    pos[ref] = np.arange(ref.size)
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))]))
    assert np.array_equal(position.cpu().numpy().reshape(-1), pos)
    assert np.array_equal(order.cpu().numpy(), np.concatenate([ref, np.full(flat.size - ref.size, -1)]))


@pytest.mark.parametrize("B", [20000, 300000])
def test_group_captured_and_replayed(B):
    """Lists of several blocks: the counts in the workspace are made anew by every replay."""
    E = 128
    ids = torch.randint(0, E, (B, 8), generator=gen(1), device="cuda", dtype=torch.int32)
    ws = torch.full((int(md.load().moe_group_workspace_bytes(B, 8, E)),), 255, dtype=torch.uint8, device="cuda")
    got = md.moe_group(ids, E, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = md.moe_group(ids, E, workspace=ws)
    for i in range(3):
        ids.copy_(torch.randint(0, E, (B, 8), generator=gen(60 + i), device="cuda", dtype=torch.int32))
        want = md.moe_group(ids, E)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_group_time_grows_with_the_slots():
    """Eight times the slots take about eight times as long, not the square of it."""
    def best(B):
        ids = torch.randint(0, 256, (B, 8), generator=gen(B), device="cuda", dtype=torch.int32)
        out = md.moe_group(ids, 256)
        ws = torch.empty(int(md.load().moe_group_workspace_bytes(B, 8, 256)), dtype=torch.uint8, device="cuda")
        times = []
        for _ in range(6):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(3):
                md.moe_group(ids, 256, order=out[0], position=out[1], offsets=out[2], workspace=ws)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end) / 3)
        return min(times)

    small, large = best(1 << 19), best((1 << 22) - 1)
    print(f"group: {small * 1e3:.0f} us and {large * 1e3:.0f} us", flush=True)
    assert large <= 16 * small


# ---------------------------------------------------------------------------- the layer with bfloat16 outputs

@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
def test_prefill_agrees_with_decode_in_bfloat16(wformat):
    """moe_prefill rounds each expert's row to bfloat16 before the weighted sum, moe_decode does not: a term is off by
    at most half a step of it. Intermediate values can differ by one step where a float32 sum lies next to a border
    (2 * 2^-8 of the result in the 2-norm allowed, as for float32 outputs), and both outputs are rounded once."""
    x, logits, mats = layer_inputs(200, 16, 4, 512, 256, wformat, 27)
    x = x.to(torch.bfloat16)
    ids, w = md.moe_route(logits, 4)
    ref = md.moe_decode(x, ids, w, *mats, inter_dtype=torch.bfloat16, wformat=wformat).double()
    out = md.moe_prefill(x, ids, w, *mats, wformat=wformat).double()
    rows = torch.zeros_like(ref)
    for j in range(4):                            # the terms, one at a time
        alone = torch.zeros_like(w)
        alone[:, j] = w[:, j]
        rows += md.moe_prefill(x, ids, alone, *mats, out_dtype=torch.float32, wformat=wformat).double().abs()
    half = 2.0 ** -8
    assert float((out - ref).norm()) <= 2 * half * float(ref.norm()) + half * float(rows.norm() + 2 * ref.norm())


# ---------------------------------------------------------------------------- MXFP8 rows on the scaled instructions

@pytest.mark.parametrize("wformat", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_prefill_fast(wformat, out_dtype):
    """The layer of the default call: where an intermediate code takes its neighbour it is an eighth of it off (2 % of
    the codes allowed: an eighth of the root of that), sums differ by what is dropped, bfloat16 rows and outputs by
    their roundings."""
    x, logits, mats = layer_inputs(700, 16, 4, 512, 256, wformat, 33)
    q, s = quantize(x)
    ids, w = md.moe_route(logits, 4)
    ref = md.moe_prefill(q, ids, w, *mats, x_s=s, out_dtype=out_dtype, wformat=wformat).double()
    out = md.moe_prefill(q, ids, w, *mats, x_s=s, out_dtype=out_dtype, wformat=wformat, fast=True).double()
    rel = float((out - ref).norm() / ref.norm())
    print(f"prefill fast {wformat} {out_dtype}: {rel:.2e}", flush=True)
    assert 0 < rel <= 0.02 ** 0.5 / 8 + (3 * 2.0 ** -8 if out_dtype == torch.bfloat16 else 0)


def test_prefill_fast_captured_and_replayed():
    x, logits, mats = layer_inputs(600, 16, 4, 256, 128, "mxfp8", 31)
    q, s = quantize(x)
    ids, w = md.moe_route(logits, 4)
    call = lambda fast: md.moe_prefill(q, ids, w, *mats, x_s=s, fast=fast)  # noqa: E731
    call(True), call(False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(True), call(False)
    for i in range(3):
        a, b = quantize(torch.randn(600, 256, generator=gen(70 + i), device="cuda"))
        q.copy_(a)
        s.copy_(b)
        want = call(True), call(False)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v), i


def test_fast_refusals():
    a = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w_q, w_s = torch.zeros(2, 32, 64, dtype=torch.uint8, device="cuda"), torch.zeros(2, 32, 2, dtype=torch.uint8, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="fast"):
        md.moe_grouped_matmul(a, off, w_q, w_s, fast=True)
    with pytest.raises(ValueError, match="fast"):
        md.moe_grouped_gate_up(a, off, w_q, w_s, w_q, w_s, fast=True)
