"""GPU tests of the dense product on the ways that the sizes of test_gpu_block.py leave out, against the same float64 results
and bounds."""
import math

import pytest
import torch

from linear_paths import MORE_SIZES, PAIRS, TYPES
from output_centric_expert_amd import moedecode as md
from test_gpu_block import ACTS, bits, check_linear, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    md.load()


@pytest.mark.parametrize("B,K,N", MORE_SIZES)
@pytest.mark.parametrize("x_type,w_type", PAIRS)
def test_linear(B, K, N, x_type, w_type):
    g = gen(B * 17 + K * 5 + N)
    x, w = randn(g, B, K).to(TYPES[x_type]), (randn(g, N, K) / math.sqrt(K)).to(TYPES[w_type])
    bias, residual = randn(g, N), randn(g, B, N).bfloat16()
    act = ACTS[(B + N) % len(ACTS)]
    check_linear(x, w, bias, act, residual, md.moe_linear(x, w, bias=bias, activation=act, residual=residual, out_dtype=torch.float32))


@pytest.mark.parametrize("B,K,N", MORE_SIZES)
@pytest.mark.parametrize("x_type,w_type", PAIRS)
def test_linear_whole_numbers(B, K, N, x_type, w_type):
    """K products of numbers up to `most` and 3 stay below 2^24: every float32 sum is exact. Float32 x holds numbers that no
    bfloat16 does."""
    g = gen(B + K * 3 + N)
    most = min(1000, (1 << 24) // (3 * K) - 1) if x_type == "f32" else 3
    x = torch.randint(-most, most + 1, (B, K), generator=g, device="cuda")
    w = torch.randint(-3, 4, (N, K), generator=g, device="cuda")
    ref = (x.double() @ w.double().T).float()
    bias, res = torch.randint(-9, 10, (N,), generator=g, device="cuda"), torch.randint(-99, 100, (B, N), generator=g, device="cuda")
    xv, wv = x.to(TYPES[x_type]), w.to(TYPES[w_type])
    out = md.moe_linear(xv, wv, bias=bias.float(), activation="relu", residual=res.bfloat16(), out_dtype=torch.float32)
    assert torch.equal(out, torch.relu(ref + bias) + res)
    # rounded outputs, the residual in their place
    out = res.bfloat16()
    want = (ref + out.float()).bfloat16()
    assert md.moe_linear(xv, wv, residual=out, out=out) is out
    assert torch.equal(bits(out), bits(want))
