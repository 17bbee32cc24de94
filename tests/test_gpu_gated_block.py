"""A gated feed-forward block's training step in block-scaled FP8, end to end, against 64
bits: every part is checked from the codes that the step itself wrote before it."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gated_reference as G
import gemm_reference as R
from fp8_scaled_quantization_gb300 import pipelines as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def make(rows, inn, hidden, experts, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    lead = () if experts is None else (experts,)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    return (rand(rows, inn).bfloat16(), (rand(*lead, 2, hidden, inn) * 1.5 / inn ** 0.5).bfloat16(),
            (rand(*lead, inn, hidden) / hidden ** 0.5).bfloat16(), (rand(rows, inn) * 1e-2).bfloat16())


def check(step, counts, fa, fg, act):
    used, ends = sum(counts), [sum(counts[:i + 1]) for i in range(len(counts))]
    stacked = lambda t, dims: t if t.dim() == dims else t[None]  # noqa: E731
    wg, sg = stacked(step.qgu, 4), stacked(step.sgu_w, 4)
    wd, sd = stacked(step.qd, 3), stacked(step.sd_w, 3)
    dgu_q, sdgu, dgu_t, sdgu_t, h_t, sh_t = step.grads
    hidden, inn = wg.shape[-2:]
    rows = step.x.shape[0]
    xv, dyv = R.values(*step.qx[:2], fa, 1), R.values(*step.qdy[:2], fg, 1)
    xc, dyc = R.values(*step.qx[2:], fa, 1), R.values(*step.qdy[2:], fg, 1)
    hv = R.values(*step.h, R.E4M3, 1)
    kept = [R.values(step.kept[0][:, i], step.kept[1][:, i], R.E4M3, 1) for i in (0, 1)]
    grads = R.values(dgu_q.view(rows, -1), sdgu.view(rows, -1), fg, 1)
    grads_c = R.values(dgu_t.view(2 * hidden, rows), sdgu_t.view(2 * hidden, -1), fg, 1)
    hc = R.values(h_t, sh_t, R.E4M3, 1)
    gu = torch.zeros((rows, 2, hidden), dtype=torch.float64, device=DEV)
    bound, wanted = torch.zeros_like(gu), {"gate_up": [], "down": []}
    for e, (a, b) in enumerate(zip([0] + ends, ends)):
        r = slice(a, b)
        w1 = [R.values(wg[e, i], sg[e, i], fa, 128) for i in (0, 1)]
        w2 = R.values(wd[e], sd[e], fa, 128)
        if b > a:
            for i in (0, 1):
                gu[r, i], bound[r, i] = R.product(xv[r], w1[i])
            R.check(step.y[r], *R.product(hv[r], w2))
            R.check(step.dh[r], *R.product(dyv[r], w2.T))
            R.check(step.dx[r], *R.product(grads[r], torch.cat(w1).T))
        # (a group may touch one block more than its length says)
        value, far = R.product(grads_c[:, r], xc[:, r])
        wanted["gate_up"].append((value, far * 2))
        value, far = R.product(dyc[:, r], hc[:, r])
        wanted["down"].append((value, far * 2))
    h, eh = G.gated(gu[:used, 0], gu[:used, 1], bound[:used, 0], bound[:used, 1], act)
    G.check_tiles(step.h[0][:used], step.h[1][:used], h, eh, R.E4M3)
    G.check_tiles(step.kept[0][:used], step.kept[1][:used], gu[:used], bound[:used], R.E4M3)
    for t in (step.y, step.dx):
        assert (t[used:] == 0).all()
    parts = G.backward(step.dh.double(), *kept, act)
    for i in (0, 1):
        G.check_tiles(dgu_q[:, i], sdgu[:, i], *parts[i], fg)
        G.check_tiles(dgu_t[i], sdgu_t[i], parts[i][0].T, parts[i][1].T, fg)
    G.check_tiles(h_t, sh_t, parts[2][0].T, parts[2][1].T, R.E4M3)
    every = wanted["gate_up"] + wanted["down"]
    norm = float(sum((v ** 2).sum() for v, _ in every).sqrt())
    # the gradients' own errors move the norm by their norm at most; the clip adds (16 + 6) * 2^-24
    rel = float(sum((b ** 2).sum() for _, b in every).sqrt()) / norm + 22 * 2.0 ** -24
    assert abs(step.norm.item() - norm) <= rel * norm
    factor = min(1.0, step.max_norm / (norm + 1e-6))
    for got, name in ((step.dgate_up, "gate_up"), (step.ddown, "down")):
        for d, (value, far) in zip(got.view(-1, *wanted[name][0][0].shape), wanted[name]):
            R.check(d, value * factor, (far + rel * value.abs()) * factor * (1 + 2.0 ** -20))


@pytest.mark.parametrize("rows,inn,hidden", [(256, 384, 256), (100, 200, 128), (5, 256, 640), (777, 512, 384)])
@pytest.mark.parametrize("act,grad_fmt", [(G.SILU, fq.E4M3), (G.GELU, fq.E5M2)])
def test_block_step(rows, inn, hidden, act, grad_fmt):
    step = P.GatedBlockStep(*make(rows, inn, hidden, None, rows), act=act, grad_fmt=grad_fmt, max_norm=0.5)
    step.run()
    torch.cuda.synchronize()
    check(step, [rows], fq.E4M3, grad_fmt, act)


@pytest.mark.parametrize("counts,spare", [([128, 256, 0, 128], 0), ([7, 300, 0, 1, 92], 0), ([40, 24], 64)])
def test_experts_step(counts, spare):
    ends = torch.tensor(counts, device=DEV).cumsum(0)
    x, gate_up, down, dy = make(sum(counts) + spare, 256, 384, len(counts), 3)
    step = P.GatedBlockStep(x, gate_up, down, dy, ends, grad_fmt=fq.E5M2, max_norm=0.1)
    step.run()
    torch.cuda.synchronize()
    check(step, counts, fq.E4M3, fq.E5M2, G.SILU)


def test_step_in_a_graph_gives_the_same():
    x, gate_up, down, dy = make(300, 256, 256, 3, 5)
    step = P.GatedBlockStep(x, gate_up, down, dy, torch.tensor([100, 200, 290], device=DEV))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step.run()
    torch.cuda.synchronize()
    outs = (step.y, step.dx, step.dgate_up, step.ddown, step.norm, *step.h, *step.kept, *step.grads)
    first = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step.run()
    for t in outs:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_gradients_follow_the_loss():
    """The step's gradients against central differences of the loss sum(y dy) in 64 bits, along
    the direction of each gradient: FP8 of every operand leaves a few percent."""
    x, gate_up, down, dy = make(512, 256, 256, None, 8)
    step = P.GatedBlockStep(x, gate_up, down, dy, max_norm=1e30)
    step.run()
    torch.cuda.synchronize()

    def loss(x, gu, d):
        g, u = x @ gu[0].T, x @ gu[1].T
        return ((g * torch.sigmoid(g) * u) @ d.T * dy.double()).sum()

    at = [t.double() for t in (x, gate_up, down)]
    for i, grad in enumerate((step.dx, step.dgate_up, step.ddown)):
        way = grad.double() / grad.double().norm()
        e = 1e-3
        ends = [loss(*[t + sign * e * way if j == i else t for j, t in enumerate(at)]) for sign in (1, -1)]
        slope = float(ends[0] - ends[1]) / (2 * e)
        # Relative noise of an E4M3 code: at most half a step, 2^-4, and about 2^-5.1 in the mean square.
        # A gradient is off by the noise of the three factors it is made of, independent from element to
        # element, which adds to its length by less than (1 + 3 * 2^-10) and turns it by less than 6%.
        assert abs(slope / float(grad.double().norm()) - 1) < 0.06
