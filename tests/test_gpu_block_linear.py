"""A layer's training step in block-scaled FP8, end to end, against 64 bits:
every product is checked from the codes that the step itself quantized."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gemm_reference as R
from fp8_scaled_quantization_gb300 import pipelines as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def make(rows, inn, out, experts, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((rows, inn), generator=g, device=DEV).bfloat16()
    dy = (torch.randn((rows, out), generator=g, device=DEV) * 1e-2).bfloat16()
    shape = (out, inn) if experts is None else (experts, out, inn)
    return x, (torch.randn(shape, generator=g, device=DEV) * 0.03).bfloat16(), dy


def check(step, counts, fa, fg):
    xv, gv = R.values(*step.qx[:2], fa, 1), R.values(*step.qdy[:2], fg, 1)
    xc, gc = R.values(*step.qx[2:], fa, 1), R.values(*step.qdy[2:], fg, 1)
    w, s = (step.qw, step.sw) if step.qw.dim() == 3 else (step.qw[None], step.sw[None])
    dw = step.dweight if step.dweight.dim() == 3 else step.dweight[None]
    norm, start, want = 0.0, 0, []
    for e, c in enumerate(counts):
        r = slice(start, start + c)
        wv = R.values(w[e], s[e], fa, 128)
        if c:
            R.check(step.y[r], *R.product(xv[r], wv))
            R.check(step.dx[r], *R.product(gv[r], wv.T))
        value, bound = R.product(gc[:, r], xc[:, r])
        want.append((value, bound * 2))  # a group may touch one block more than its length says
        norm += (value ** 2).sum()
        start += c
    assert (step.y[start:] == 0).all() and (step.dx[start:] == 0).all()
    norm = float(norm.sqrt())
    # the gradients' own errors move the norm by their norm at most; the clip adds (16 + 6) * 2^-24
    rel = float(sum((b ** 2).sum() for _, b in want).sqrt()) / norm + 22 * 2.0 ** -24
    assert abs(step.norm.item() - norm) <= rel * norm
    factor = min(1.0, step.max_norm / (norm + 1e-6))
    for e, (value, bound) in enumerate(want):
        R.check(dw[e], value * factor, (bound + rel * value.abs()) * factor * (1 + 2.0 ** -20))


@pytest.mark.parametrize("rows,inn,out", [(256, 512, 384), (100, 256, 130), (1000, 640, 768)])
@pytest.mark.parametrize("grad_fmt", [fq.E4M3, fq.E5M2])
def test_layer_step(rows, inn, out, grad_fmt):
    x, w, dy = make(rows, inn, out, None, rows)
    step = P.BlockLinearStep(x, w, dy, grad_fmt=grad_fmt, max_norm=0.5)
    step.run()
    torch.cuda.synchronize()
    check(step, [rows], fq.E4M3, grad_fmt)


@pytest.mark.parametrize("counts,spare", [([128, 256, 0, 128], 0), ([7, 300, 0, 1, 92], 0), ([40, 24], 64)])
def test_experts_step(counts, spare):
    rows, inn, out = sum(counts) + spare, 384, 256
    x, w, dy = make(rows, inn, out, len(counts), rows)
    ends = torch.tensor(counts, device=DEV).cumsum(0)
    step = P.BlockLinearStep(x, w, dy, ends, grad_fmt=fq.E5M2, max_norm=0.1)
    step.run()
    torch.cuda.synchronize()
    check(step, counts, fq.E4M3, fq.E5M2)


def test_step_in_a_graph_gives_the_same():
    x, w, dy = make(384, 512, 256, 3, 5)
    ends = torch.tensor([100, 200, 384], device=DEV)
    step = P.BlockLinearStep(x, w, dy, ends)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step.run()
    torch.cuda.synchronize()
    first = [t.clone() for t in (step.y, step.dx, step.dweight, step.norm)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step.run()
    for t in (step.y, step.dx, step.dweight, step.norm):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (step.y, step.dx, step.dweight, step.norm)))
