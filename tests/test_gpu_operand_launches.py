"""Launches of a product by how many of its operands have to be copied to aligned rows: one more
for one or for both."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gated_reference as G
import gemm_reference as R
import test_gpu_gated as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def launches(call):
    before = fq.launch_count()
    call()
    return fq.launch_count() - before


def at(t, shift):
    moved = T.Out(t.shape, shift=shift)
    moved.t.copy_(t)
    return moved.t


# k a multiple of 16: an operand is copied where it starts off 16 bytes
@pytest.mark.parametrize("m", [3, 40, 300])
@pytest.mark.parametrize("odd", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_starts(m, odd):
    n, k = 300, 400
    a, sa, b, sb = T.operands(m, n, k, 1)
    a, b = at(a, odd[0]), at(b, odd[1])
    outs = T.outputs(m, n, True)
    assert launches(lambda: fq.fp8_gemm_block_gated(a, sa, b, sb, *[o.t for o in outs])) == 1 + any(odd)
    T.check(outs, *T.projections(a, sa, b, sb), G.SILU)
    d = torch.empty((m, n), device=T.DEV)
    assert launches(lambda: fq.fp8_gemm_block(a, sa, b[0], sb[0], d)) == 1 + any(odd)
    R.check(d, *R.product(R.values(a, sa, R.E4M3, 1), R.values(b[0], sb[0], R.E4M3, 128)))


@pytest.mark.parametrize("m", [3, 40, 300])
def test_odd_rows(m):
    ops = T.operands(m, 300, 401, 2)
    outs = T.outputs(m, 300, False)
    assert launches(lambda: fq.fp8_gemm_block_gated(*ops, *[o.t for o in outs])) == 2
    ends = torch.tensor([m - 1, m], device=T.DEV)
    ops = T.operands(m, 300, 401, 2, 2)
    assert launches(lambda: fq.fp8_gemm_block_gated_grouped(*ops, ends, *[o.t for o in outs])) == 2
    T.grouped_check(ops, [m - 1, 1], outs, G.SILU)
