"""The gated block with operands of both formats on both sides, dense and per expert."""
from __future__ import annotations

import math

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gated_bounds as B
import gated_reference as G
import gemm_reference as R
import test_gpu_gated as T
import test_gpu_gated_block as S
from fp8_scaled_quantization_gb300 import pipelines as P

pytestmark = pytest.mark.gpu
FORMATS = [(R.E4M3, R.E5M2), (R.E5M2, R.E4M3), (R.E5M2, R.E5M2)]


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def operands(m, n, k, seed, fmt_a, fmt_b, experts=None, size=2.0):
    """Codes over the whole range of each format; projections of about `size`."""
    g, kb, nb = T.gen(seed), G.blocks(k), G.blocks(n)
    lead = () if experts is None else (experts,)
    rms = [R.decode_table(f)[torch.arange(0x7F if f == R.E4M3 else 0x7C)].square().mean().sqrt().item() for f in (fmt_a, fmt_b)]
    a, b = R.finite_codes((m, k), fmt_a, g, T.DEV), R.finite_codes((*lead, 2, n, k), fmt_b, g, T.DEV)
    sa = torch.exp(torch.randn((m, kb), generator=g, device=T.DEV) * 0.5) / rms[0]
    sb = torch.exp(torch.randn((*lead, 2, nb, kb), generator=g, device=T.DEV) * 0.3) / rms[1] * size / math.sqrt(k)
    return a, sa, b, sb


@pytest.mark.parametrize("fmt_a,fmt_b", FORMATS)
@pytest.mark.parametrize("m,n,k", [(1, 512, 1024), (7, 130, 300), (24, 1030, 400), (60, 2048, 1152), (300, 640, 1040),
                                   (2000, 1300, 515)])
def test_dense(m, n, k, fmt_a, fmt_b):
    ops = operands(m, n, k, m + n, fmt_a, fmt_b)
    for keep, act in ((True, G.SILU), (False, G.GELU)):
        outs = T.outputs(m, n, keep)
        fq.fp8_gemm_block_gated(*ops, *[o.t for o in outs], fmt_a=fmt_a, fmt_b=fmt_b, act=act)
        B.check_forward([o.t for o in outs], *T.projections(*ops, fmt_a, fmt_b), act)
        assert all(o.intact() for o in outs)


@pytest.mark.parametrize("fmt_a,fmt_b", FORMATS)
@pytest.mark.parametrize("counts,spare,n,k", [([5, 0, 12, 1], 3, 256, 384), ([300, 0, 129, 1, 255], 13, 520, 300),
                                              ([40] * 6, 0, 300, 1040)])
def test_experts(counts, spare, n, k, fmt_a, fmt_b):
    rows, used = sum(counts) + spare, sum(counts)
    a, sa, b, sb = operands(rows, n, k, rows, fmt_a, fmt_b, len(counts))
    ends = torch.tensor(counts, device=T.DEV).cumsum(0)
    for keep, act in ((True, G.GELU), (False, G.SILU)):
        outs = T.outputs(rows, n, keep)
        fq.fp8_gemm_block_gated_grouped(a, sa, b, sb, ends, *[o.t for o in outs], fmt_a=fmt_a, fmt_b=fmt_b, act=act)
        start = 0
        for e, c in enumerate(counts):
            r = slice(start, start + c)
            if c:
                B.check_forward([o.t[r] for o in outs], *T.projections(a[r], sa[r], b[e], sb[e], fmt_a, fmt_b), act)
            start += c
        assert all(not (o.t[used:] & 0x7F).any() for o in outs[::2]) and all((o.t[used:] == 1).all() for o in outs[1::2])
        assert all(o.intact() for o in outs)


@pytest.mark.parametrize("m,k", [(2, 0), (20, 0), (300, 0)])
def test_no_contraction_in_wide_rows(m, k):
    """Rows that are multiples of 16 bytes, also fewer of them than a store's 32."""
    n = 384
    outs = T.outputs(m, n, True)
    empty = [torch.empty(s, dtype=d, device=T.DEV) for s, d in (((m, k), torch.uint8), ((m, 0), torch.float32),
                                                                ((2, n, k), torch.uint8), ((2, 3, 0), torch.float32))]
    fq.fp8_gemm_block_gated(*empty, *[o.t for o in outs])
    assert all(not (o.t & 0x7F).any() for o in outs[::2]) and all((o.t == 1).all() for o in outs[1::2])
    assert all(o.intact() for o in outs)


@pytest.mark.parametrize("fmt,grad_fmt", [(fq.E5M2, fq.E5M2), (fq.E5M2, fq.E4M3)])
def test_block_step(fmt, grad_fmt):
    step = P.GatedBlockStep(*S.make(300, 384, 256, None, 2), fmt=fmt, grad_fmt=grad_fmt, max_norm=0.5)
    step.run()
    torch.cuda.synchronize()
    S.check(step, [300], fmt, grad_fmt, G.SILU)


def test_experts_step():
    counts = [7, 300, 0, 1, 92]
    x, gate_up, down, dy = S.make(sum(counts) + 20, 256, 384, len(counts), 3)
    step = P.GatedBlockStep(x, gate_up, down, dy, torch.tensor(counts, device=T.DEV).cumsum(0), fmt=fq.E5M2, act=fq.ACT_GELU_TANH,
                            grad_fmt=fq.E5M2, max_norm=0.1)
    step.run()
    torch.cuda.synchronize()
    S.check(step, counts, fq.E5M2, fq.E5M2, G.GELU)
