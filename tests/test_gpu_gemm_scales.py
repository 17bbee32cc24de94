"""The order in which a product's scales are applied, at scales whose products leave the
fp32 range.  Codes and scales are powers of two, and only the first block of 128 steps
has codes, so that every step of the formula is exact but for overflow and underflow:
  128 x 128 blocks of B   (sa * sb) * P
  1 x 128 tiles of B      (P * sb) * sa
The result must be the same bits whichever kernel the sizes select."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
K = 4096  # long enough for every kernel to be chosen at some m


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def code(exponent):
    """E4M3 code of 2^exponent, -6 .. 8; smaller ones, down to 2^-9, are subnormal."""
    return (exponent + 7) << 3 if exponent >= -6 else 1 << (exponent + 9)


def operand(rows, exponent, zero_rows):
    q = torch.zeros((rows, K), dtype=torch.uint8, device=DEV)
    q[:, :128] = code(exponent)
    q[zero_rows] = 0
    return q, (q != 0).double() * 2.0 ** exponent


def factors(rows, exponent):
    """The first block's scale; those of the blocks without codes are 1."""
    s = torch.ones((rows, K // 128), device=DEV)
    s[:, 0] = 2.0 ** exponent
    return s


# exponents of: A's codes, B's codes, A's scales, B's scales.  P is 2^(a + b + 7).
CASES = [
    (8, 8, -80, -80),    # sa * sb underflows to 0, the result is 2^-137
    (8, 8, -100, -40),   # sa * sb is subnormal
    (-9, -9, 90, 60),    # sa * sb overflows, the result is 2^139
    (-9, -9, 80, 50),    # ... is 2^119
    (8, 8, -20, 110),    # P * sb overflows
    (0, 0, -3, 4),
]


@pytest.mark.parametrize("a_exp,b_exp,sa_exp,sb_exp", CASES)
@pytest.mark.parametrize("form", ["nk", "kn", "tiles", "grouped tiles"])
def test_scales_outside_the_fp32_range(form, a_exp, b_exp, sa_exp, sb_exp):
    n = 2064
    for m in (1, 16, 20, 64, 100, 128, 300, 2000):
        a, av = operand(m, a_exp, [0] if m > 1 else [])
        b, bv = operand(n, b_exp, [3])
        sa, sb = factors(m, sa_exp), factors(n if "tiles" in form else -(-n // 128), sb_exp)
        p = (av @ bv.T).float()
        want = (p * sb[0, 0]) * sa[0, 0] if "tiles" in form else p * (sa[0, 0] * sb[0, 0])
        d = torch.empty((m, n), device=DEV)
        if form == "grouped tiles":
            d = torch.empty((1, m, n), device=DEV)
            fq.fp8_gemm_block_grouped_wgrad(a, sa, b, sb, torch.tensor([K], device=DEV), d)
            d = d[0]
        elif form == "kn":
            fq.fp8_gemm_block(a, sa, b.T.contiguous(), sb.T.contiguous(), d, b_layout=fq.B_KN)
        else:
            fq.fp8_gemm_block(a, sa, b, sb, d, b_block_rows=1 if form == "tiles" else 128)
        same = (d == want) | (d.isnan() & want.isnan())
        assert same.all(), (m, d[~same][:4], want[~same][:4])
