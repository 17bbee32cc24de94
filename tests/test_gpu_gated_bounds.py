"""The gated block where the sigmoid saturates or is flat, with bounds that stay far below the values there."""
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


@pytest.mark.parametrize("size", [1e-6, 2.0, 30.0, 1e4])
@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("m,n,k", [(9, 384, 512), (30, 400, 384), (60, 384, 512), (300, 384, 512), (280, 515, 700)])
def test_projections_of_all_sizes(m, n, k, act, size):
    ops = T.operands(m, n, k, m + 1, size=size)
    outs = T.outputs(m, n, True)
    fq.fp8_gemm_block_gated(*ops, *[o.t for o in outs], act=act)
    gu, bound = T.projections(*ops)
    B.check_forward([o.t for o in outs], gu, bound, act)
    h, eh = B.gated(gu[:, 0], gu[:, 1], bound[:, 0], bound[:, 1], act)
    assert B.loose(h, eh, R.E4M3) < 0.05


@pytest.mark.parametrize("size", [1e-30, 1e-4, 1.0, 30.0, 1e4, 1e6])
@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("dtype,fmt", [(torch.float32, R.E5M2), (torch.float32, R.E4M3), (torch.bfloat16, R.E4M3)])
def test_backward_of_projections_of_all_sizes(act, size, dtype, fmt):
    for rows, n in ((200, 384), (131, 517)):
        dh = torch.randn((rows, n), generator=T.gen(1), device=T.DEV).to(dtype)
        gu, sgu = T.checkpoint(rows, n, 2, size)
        outs = T.gradient_outputs(rows, n)
        T.back(dh, gu, sgu, outs, act=act, fmt_grad=fmt)
        B.check_backward([o.t for o in outs], dh, gu, sgu, act, fmt)
        g, u = (R.values(gu[:, i], sgu[:, i], R.E4M3, 1) for i in (0, 1))
        if size > 1e-30:  # (products of 1e-60 are zeros)
            assert all(B.loose(v, e, fmt) < 0.01 for v, e in B.backward(dh.double(), g, u, act))
