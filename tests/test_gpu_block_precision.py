"""GPU tests of the last bits of the operators around the MoE block: float32 operands of the dense product, value for value,
and the activations by their relative error, in their tails and next to zero too."""
import math

import pytest
import torch

from linear_paths import MORE_SIZES
from output_centric_expert_amd import moedecode as md
from test_gpu_block import bits, gen, randn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
WITH_F32 = [("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")]
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# of one row, of few rows (either side, 16 and 32), of tiles, with k whole and split
SIZES = [(1, 200, 90), (2, 77, 5), (5, 512, 300), (16, 7168, 256), (40, 65, 40), (64, 7168, 256), (300, 77, 500), (700, 4096, 900),
         (1000, 1111, 777), (3000, 200, 20), (200, 20000, 40)] + MORE_SIZES[::3]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    md.load()


def one_hot(g, rows, K):
    """[rows, K] with a one in a random place of each row, and the places."""
    at = torch.randint(0, K, (rows,), generator=g, device="cuda")
    t = torch.zeros(rows, K, device="cuda")
    t[torch.arange(rows, device="cuda"), at] = 1.0
    return t, at


# ---------------------------------------------------------------------------- float32 operands

@pytest.mark.parametrize("B,K,N", SIZES)
@pytest.mark.parametrize("x_type,w_type", WITH_F32)
def test_every_bit_of_a_float32_operand(B, K, N, x_type, w_type):
    """The other side selects one value for each output: all of its 24 bits come through. A value's parts add up to it without
    a rounding (from the lowest: each sum is a tail of the value), everything else adds zeros."""
    g = gen(B + K + N)
    if x_type == "f32":
        x, (w, at) = randn(g, B, K), one_hot(g, N, K)
        out = md.moe_linear(x, w.to(TYPES[w_type]), out_dtype=torch.float32)
        assert torch.equal(bits(out), bits(x[:, at].contiguous()))
    if w_type == "f32":
        w, (x, at) = randn(g, N, K), one_hot(g, B, K)
        out = md.moe_linear(x.to(TYPES[x_type]), w, out_dtype=torch.float32)
        assert torch.equal(bits(out), bits(w[:, at].T.contiguous()))


@pytest.mark.parametrize("B,K,N", SIZES)
def test_products_of_lower_parts(B, K, N):
    """12 times 12 bits: whole numbers that two parts hold, of both sides. Their product and its sums in between are whole
    numbers up to 2^24: exact."""
    g = gen(B * 3 + K + N)
    x = torch.randint(-4095, 4096, (B, K), generator=g, device="cuda").float()
    w, at = one_hot(g, N, K)
    scale = torch.randint(1, 4096, (N,), generator=g, device="cuda").float()
    out = md.moe_linear(x, w * scale[:, None], out_dtype=torch.float32)
    assert torch.equal(out, x[:, at] * scale)


@pytest.mark.parametrize("B", [1, 3, 40, 300])
@pytest.mark.parametrize("x_type,w_type", WITH_F32)
def test_tiny_float32_operands(B, x_type, w_type):
    """A part below 2^-126 is a bfloat16 in steps of 2^-133: a float32 value of 2^-110 and more (steps of 2^-133 at least) keeps
    all of its bits, a smaller one is off by at most half such a step. One row is exact."""
    g = gen(B)
    K, N = 64, 80
    rows, other = (B, N) if x_type == "f32" else (N, B)
    v = torch.ldexp(1 + torch.rand(rows, K, generator=g, device="cuda"),
                    torch.randint(-149, -100, (rows, K), generator=g, device="cuda"))
    sel, at = one_hot(g, other, K)
    if x_type == "f32":
        out = md.moe_linear(v, sel.to(TYPES[w_type]), out_dtype=torch.float32)
        want = v[:, at]
    else:
        out = md.moe_linear(sel.to(TYPES[x_type]), v, out_dtype=torch.float32)
        want = v[:, at].T
    off = (out.double() - want.double()).abs()
    assert (off <= (0.0 if B == 1 else 2.0 ** -134)).all()
    assert (off[want >= 2.0 ** -110] == 0).all()


# ---------------------------------------------------------------------------- activations

def arguments():
    dense = torch.linspace(-110, 110, 1 << 17, dtype=torch.float64).float()
    far = torch.exp2(torch.linspace(-100, 7, 1 << 15, dtype=torch.float64)).float()
    border = (torch.tensor(0.25).view(torch.int32) + torch.arange(-4096, 4097, dtype=torch.int32)).view(torch.float32)
    return torch.cat([dense, far, -far, border, -border]).cuda()


def activation(v, act):
    """(float64 value, bound of the float32 one's error). U is half of a last place, 2^-24 of a value. The hardware's exp2 and
    reciprocal are off by a last place (2 U) each, the constant log2(e) by 0.23 U of itself, every operation by U.

    sigmoid: the exponent's two roundings are 1.23 |v| U of exp(-v); with exp2's 2, the sum's 1 and the reciprocal's 2 of the
      result. Below 2^-126 the reciprocal is 0.
    silu: one product more; what the sigmoid loses below 2^-126, times v.
    gelu: erfc(z) at z = -v / sqrt 2, two roundings that are 1.3 U of z. |z erfc'(z) / erfc(z)| is at most 2 z^2 + 1 = v^2 + 1
      (for z > 0 as erfc(z) >= 2/sqrt(pi) exp(-z^2) / (z + sqrt(z^2 + 2)); below 1/2 for z < 0). erfc itself: 16 last places,
      the worst that OpenCL allows, and 0 below 2^-126.
    gelu_tanh: u's outer constant is off by 0.78 U and its product and sum by 1 each, the inner constant by 0.58 and its two
      products by 1 each: 6 U at most. The sigmoid of u is then off by (1.23 + 6) |u| + 5, the last product by 1.
    tanh: up to 0.25 v + v^3 P: one rounding of the sum, v^3 P is at most 2 % of it and off by 6 U, Taylor's series ends 0.14 U
      off. Beyond, (1 - e) / (1 + e) with e = exp(-2v): e's error of 2.46 |v| + 2 U counts 1 / sinh(2 |v|) times, 5.0 at
      0.25 and less behind; differences, quotient and product 5."""
    x = v.double()
    a, e = x.abs(), torch.exp(-x)
    least = 2.0 ** -126
    if act == "sigmoid":
        ref = 1 / (1 + e)
        return ref, (1.23 * a + 5) * U * ref + least
    if act == "silu":
        ref = x / (1 + e)
        return ref, (1.23 * a + 6) * U * ref.abs() + a * least
    if act == "gelu":
        ref = 0.5 * x * torch.special.erfc(-x / math.sqrt(2))
        return ref, (1.3 * (a * a + 1) + 34) * U * ref.abs() + a * least
    if act == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)
        ref = x / (1 + torch.exp(-u))
        return ref, (7.23 * u.abs() + 6) * U * ref.abs() + a * least
    if act == "tanh":
        ref = torch.tanh(x)
        return ref, torch.where(a < 0.25, 1.3, 10.1) * U * ref.abs()
    return torch.relu(x), torch.zeros_like(x)


def close(out, ref, tol):
    # (1 + U)^n is more than 1 + nU by less than a thousandth for the bounds here
    off = (out.double() - ref).abs()
    assert (off <= 1.001 * tol).all(), float((off / tol).nan_to_num(0).max())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "sigmoid", "tanh"])
@pytest.mark.parametrize("B", [1, 3, 40])
def test_activations(B, act):
    """The kernels of one row, of few rows and of tiles; the product is with one."""
    v = arguments()
    out = md.moe_linear(torch.ones(B, 1, device="cuda"), v[:, None], activation=act, out_dtype=torch.float32)
    close(out[B - 1], *activation(v, act))
    assert torch.equal(bits(out[0]), bits(out[B - 1]))


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("H", [2048, 2051])
def test_gates(H, act):
    """A gate of each value on y = 1 and a residual of 0: residual_out is the activation, by channel and by value."""
    v = arguments()
    v = v[:len(v) // H * H].view(-1, H)
    ref, tol = activation(v, act)
    one, zero = torch.ones_like(v), torch.zeros_like(v)
    close(md.moe_post_norm(one, zero, gate=v, gate_act=act)[1], ref, tol)
    first = v[:1].clone()
    close(md.moe_post_norm(one[:2], zero[:2], gate=first[0], gate_act=act)[1][1:], ref[:1], tol[:1])
    token = v.view(-1)[:4096, None].contiguous()
    out = md.moe_post_norm(torch.ones(4096, 8, device="cuda"), torch.zeros(4096, 8, device="cuda"), gate=token, gate_act=act)[1]
    close(out[:, 7], ref.view(-1)[:4096], tol.view(-1)[:4096])
