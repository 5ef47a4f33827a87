"""Host-side checks of the prompt-side calls at the ends of their ranges (no GPU needed; the addresses are never
read)."""
import os
import re
import subprocess

import pytest

from output_centric_expert_amd import moedecode as md
from test_abi import A, lib  # noqa: F401
from test_abi_prompt import gate_up, matmul, norm, prefill


@pytest.mark.parametrize("rows,K,below,above", [(md.MOED_ROWS_BF16, 2880, 700_000, 800_000),
                                                (md.MOED_ROWS_MXFP8, 1056, 4_000_000, 4_100_000)])
def test_workspace_of_rows_in_place_past_4_gib(lib, rows, K, below, above):  # noqa: F811
    """Without an order rows may take 4 GiB and more, and the workspace query answers for them too."""
    size = 2 if rows == md.MOED_ROWS_BF16 else 1
    assert below * K * size < 1 << 32 <= above * K * size
    row = (K // 32 + 15) // 16 * 16
    for n_a in (below, above):
        for matrices in (1, 2):
            need = lib.moe_grouped_workspace_bytes(8, K, 64, n_a, rows, matrices)
            assert need == (8 * 64 * matrices + (n_a if rows == md.MOED_ROWS_MXFP8 else 0)) * row, n_a
    kw = {"rows": rows, "a_s": A if rows == md.MOED_ROWS_MXFP8 else None, "n_a": above, "K": K}
    need = lib.moe_grouped_workspace_bytes(8, K, 64, above, rows, 1)
    assert matmul(lib, order=None, R=above, wsp=A, wsb=need - 1, **kw) == md.MOED_ERR_WORKSPACE
    # gathered rows of that size are refused
    assert matmul(lib, R=16, **kw) == md.MOED_ERR_SHAPE


def test_norm_refuses_one_buffer_for_two_outputs(lib):  # noqa: F811
    """Both `out` and `residual_out` may be x or the residual, but not the same one."""
    assert norm(lib) == md.MOED_ERR_SHAPE
    assert norm(lib, B=0) == md.MOED_OK


LIMITS = r"""
#include <cstdio>
#include "lds_limits.h"
static moed::LdsLimits t;
static char kernels[N + 1];
int main()
{
    for (int d = 0; d < moed::LdsLimits::kDevices; ++d)
        for (int k = 0; k < N; ++k) {
            int* have = t.find(&kernels[k], d);
            if (!have || *have)
                return printf("kernel %d on device %d: %s\n", k, d, have ? "not new" : "no room");
            *have = 1 + k * 100 + d;
        }
    for (int d = 0; d < moed::LdsLimits::kDevices; ++d)
        for (int k = 0; k < N; ++k) {
            int* have = t.find(&kernels[k], d);
            if (!have || *have != 1 + k * 100 + d)
                return printf("kernel %d on device %d is forgotten\n", k, d);
        }
    return N == moed::LdsLimits::kKernels && t.find(&kernels[N], 0) ? printf("more than all\n") : 0;
}
"""


def test_lds_limits_of_every_kernel_on_every_device(lib, tmp_path):  # noqa: F811
    """The table of LDS sizes holds each kernel that asks for one, on each device."""
    names = subprocess.run(["nm", "-C", md.LIB_PATH], capture_output=True, text=True, check=True).stdout
    asking = len(re.findall(r"__device_stub__(?:moe_product_tiled|moe_group_place|moe_gate_up_grouped_wide|"
                            r"moe_down_expert)_kernel", names))
    assert 0 < asking < 256
    csrc = os.path.join(os.path.dirname(md.LIB_PATH), "csrc")
    for n in (asking, 256):
        src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
        src.write_text(LIMITS)
        subprocess.run(["g++", "-std=c++17", f"-DN={n}", "-I", csrc, str(src), "-o", str(exe)], check=True)
        done = subprocess.run([str(exe)], capture_output=True, text=True)
        assert done.returncode == 0, done.stdout


def test_fast_rows(lib):  # noqa: F811
    """The fast form of MXFP8 rows is checked as MXFP8 rows are, and is no kind of output."""
    fast = md.MOED_ROWS_MXFP8_FAST
    for call in (gate_up, matmul):
        assert call(lib, rows=fast) == md.MOED_ERR_NULL
        assert call(lib, rows=fast, a_s=A, R=0) == md.MOED_OK
        assert call(lib, rows=fast, a_s=A, K=64) == md.MOED_ERR_NULL
        assert call(lib, out_rows=fast) == md.MOED_ERR_DTYPE
    assert prefill(lib, rows=fast) == md.MOED_ERR_NULL
    assert prefill(lib, rows=fast, x_s=A, wsb=16) == md.MOED_ERR_WORKSPACE
    for args in ((8, 64, 32, 5), (8, 512, 32, 5), (4, 1120, 64, 1000)):
        for two in (1, 2):
            assert (lib.moe_grouped_workspace_bytes(*args, fast, two) ==
                    lib.moe_grouped_workspace_bytes(*args, md.MOED_ROWS_MXFP8, two))
    assert (lib.moe_prefill_workspace_bytes(2, 8, 2, 64, 32, fast, 1) ==
            lib.moe_prefill_workspace_bytes(2, 8, 2, 64, 32, md.MOED_ROWS_MXFP8, 1) > 0)
