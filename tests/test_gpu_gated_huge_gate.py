"""A gate so large that products with it leave fp32 where the derivative does not: act' is 1 above it and 0 below."""
from __future__ import annotations

import pytest
import torch

import gated_bounds as B
import gated_reference as G
import gemm_reference as R
import test_gpu_gated as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def in_fp32(value, bound):
    """Products are taken in fp32: one beyond its largest value by more than half a step is Inf.
    (None of these inputs' lies so close to it that its bound leaves that open.)"""
    top = float(torch.finfo(torch.float32).max)
    over = value.abs() > top * (1 + 2.0 ** -25)
    assert ((value.abs() - top).abs() > bound).all()
    return torch.where(over, value.sign() * float("inf"), value), torch.where(over, 0.0, bound)


@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("dtype,fmt", [(torch.float32, R.E4M3), (torch.bfloat16, R.E5M2)])
@pytest.mark.parametrize("rows,n", [(200, 384), (131, 517)])
def test_backward(rows, n, act, dtype, fmt):
    """Gates up to 3e38 in every third row (some of h leave fp32 there); the rest stays usual, in the
    same column tiles."""
    dh = (torch.randn((rows, n), generator=T.gen(1), device=T.DEV) * 1e-3).to(dtype)
    gu, sgu = T.checkpoint(rows, n, 2)
    sgu[::3, 0] = 6e35
    assert R.values(gu[:, 0], sgu[:, 0], R.E4M3, 1).abs().max() > 2e38
    outs = T.gradient_outputs(rows, n)
    T.back(dh, gu, sgu, outs, act=act, fmt_grad=fmt)
    g, u = (R.values(gu[:, i], sgu[:, i], R.E4M3, 1) for i in (0, 1))
    parts = [in_fp32(*part) for part in B.backward(dh.double(), g, u, act)]
    assert parts[2][0].isinf().any() and all(v.isfinite().all() for v, _ in parts[:2])
    for i in (0, 1):
        G.check_tiles(outs[0].t[:, i], outs[1].t[:, i], *parts[i], fmt)
        G.check_tiles(outs[2].t[i], outs[3].t[i], parts[i][0].T, parts[i][1].T, fmt)
    G.check_tiles(outs[4].t, outs[5].t, parts[2][0].T, parts[2][1].T, R.E4M3)
    assert all(o.intact() for o in outs)
