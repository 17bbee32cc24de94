"""Outputs of the gated block's forward call beyond 2^31 and 2^32 bytes, by both kernels."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gated_bounds as B
import gated_reference as G
import gemm_reference as R
import test_gpu_gated as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def filled(m, n):
    nb = G.blocks(n)
    return [torch.full(s, 0x39, dtype=torch.uint8, device=T.DEV) if i % 2 == 0 else torch.zeros(s, device=T.DEV)
            for i, s in enumerate(((m, n), (m, nb), (m, 2, n), (m, 2, nb)))]


@pytest.mark.parametrize("m,n", [(70016, 65536), (66001, 65537)])
def test_many_rows(m, n):
    """Codes that leave by bulk copies, and ones that start anywhere (pair kernel)."""
    a, sa, b, sb = T.operands(m, n, 16, 1)
    outs = filled(m, n)
    fq.fp8_gemm_block_gated(a, sa, b, sb, *outs)
    # around 2^31 and 2^32 bytes of the projections (row 2^14 and 2^15) and of h, and both ends
    for lo in (0, 2 ** 14 - 100, 2 ** 15 - 100, 2 ** 16 - 100, m - 200):
        r = slice(lo, lo + 200)
        B.check_forward([o[r] for o in outs], *T.projections(a[r], sa[r], b, sb), G.SILU)
    assert all((o[at] > 0).all() for o in outs[1::2] for at in range(0, m, 997))


def test_many_columns():
    """16 rows of 2^28 columns and some (stream kernel): weights of zeros but in the last columns and
    some in between."""
    m, n, k = 16, 2 ** 28 + 200, 16
    nb, g = G.blocks(n), T.gen(1)
    a, sa = R.finite_codes((m, k), R.E4M3, g, T.DEV), torch.full((m, 1), 0.01, device=T.DEV)
    b, sb = torch.zeros((2, n, k), dtype=torch.uint8, device=T.DEV), torch.full((2, nb, 1), 0.01, device=T.DEV)
    spots = [(lo // 128 * 128, min(lo // 128 * 128 + 1024, n)) for lo in (0, 2 ** 26, 2 ** 27 - 512, n - 1000)]
    for lo, hi in spots:
        b[:, lo:hi] = R.finite_codes((2, hi - lo, k), R.E4M3, g, T.DEV)
    outs = filled(m, n)
    fq.fp8_gemm_block_gated(a, sa, b, sb, *outs)
    for lo, hi in spots:
        c, cb = slice(lo, hi), slice(lo // 128, -(-hi // 128))
        gu, bound = T.projections(a, sa, b[:, c], sb[:, cb])
        B.check_forward([outs[0][:, c], outs[1][:, cb], outs[2][..., c], outs[3][..., cb]], gu, bound, G.SILU)
    for lo in (2 ** 25, 2 ** 27 + 2 ** 20, n // 2 // 128 * 128, n - 10 ** 6 // 128 * 128):
        c, cb = slice(lo, lo + 4096), slice(lo // 128, lo // 128 + 32)
        if not any(a < lo + 4096 and lo < b for a, b in spots):
            assert not (outs[0][:, c] & 0x7F).any() and not (outs[2][..., c] & 0x7F).any()
            assert (outs[1][:, cb] == 1).all() and (outs[3][..., cb] == 1).all()
