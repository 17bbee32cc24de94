"""The bounds of the gated activation themselves: they hold for fp32 evaluations with the worst
approximations, and they are small against the values."""
from __future__ import annotations

import math

import pytest
import torch

import gated_bounds as B
import gated_reference as G
import gemm_reference as R

LOG2E, TWO_C, CUBE = 1.4426950408889634, 1.5957691216057308, 0.044715


def evaluate(g, act, gen):
    """act and act' in fp32 steps; the exponential and the reciprocal off by up to two units."""
    f = lambda v: torch.tensor(v, dtype=torch.float32)  # noqa: E731

    def off(t):  # to fp32 with a relative error of 2^-22 at most, which it often has
        r = (torch.rand(t.shape, generator=gen, dtype=torch.float64) * 4 - 2).clamp(-1, 1)
        return (t * (1 + (2.0 ** -22 - 2.0 ** -24) * r)).float()

    fma = lambda x, y, z: (x.double() * y.double() + z.double()).float()  # noqa: E731
    if act == G.SILU:
        t, dy = g * f(-LOG2E), torch.ones_like(g)
    else:
        c = g.clamp(-32, 32)
        c2 = c * c
        t = c * fma(c2, f(-LOG2E * TWO_C * CUBE), f(-LOG2E * TWO_C))
        dy = fma(c2, f(3 * TWO_C * CUBE), f(TWO_C))
    total = 1 + off(torch.exp2(t.double()))
    s = torch.where(total == 1, total, off(1 / total.double()))
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    a, rest = g * s, 1 - s
    return a, fma(a, rest * dy, s)


@pytest.mark.parametrize("act", [G.SILU, G.GELU])
def test_bounds_hold(act):
    gen = torch.Generator().manual_seed(1)
    g = torch.cat([torch.linspace(-100, 100, 400001), torch.linspace(-6, 6, 400001), torch.linspace(-1.5, -0.7, 100001),
                   10 ** torch.linspace(-40, 37, 10001), -10 ** torch.linspace(-40, 37, 10001), torch.zeros(2)]).float()
    a, slope, ea, es = B.activation(g.double(), act, torch.zeros(len(g), dtype=torch.float64))
    for _ in range(4):
        got_a, got_slope = evaluate(g, act, gen)
        assert ((got_a.double() - a).abs() <= ea).all()
        assert ((got_slope.double() - slope).abs() <= es).all()
    # (no more than some units in the last place of 1, or of the value)
    assert (es <= 2.0 ** -16).all() and (ea <= a.abs() * 2.0 ** -14 + 2e-36).all()


@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("share", [1e-7, 1e-3, 0.3])
def test_bounds_hold_for_a_gate_that_is_nearly_known(act, share):
    g = torch.cat([torch.linspace(-60, 60, 200001, dtype=torch.float64), 10 ** torch.linspace(-30, 37, 10001, dtype=torch.float64),
                   -10 ** torch.linspace(-30, 37, 10001, dtype=torch.float64)])
    eg = g.abs() * share
    a, slope, ea, es = B.activation(g, act, eg)
    for w in (-1.0, -0.5, 0.7, 1.0):
        near = g + w * eg
        if share < 1e-6:
            near = near.float().double()
            near = torch.where((near - g).abs() <= eg, near, g.float().double())
        got_a, got_slope = G.activation(near, act)[:2]
        # (in 64 bits act' has roundings of 1 of its own)
        assert ((got_a - a).abs() <= ea * (1 + 1e-9) + 1e-300).all()
        assert ((got_slope - slope).abs() <= es * (1 + 1e-9) + 1e-15).all()


@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("size", [1e-4, 1.0, 30.0, 1e4, 1e6, 1e30])
def test_backward_bounds_are_small(act, size):
    gen = torch.Generator().manual_seed(3)
    codes = R.finite_codes((200, 2, 384), R.E4M3, gen, "cpu")
    factors = torch.exp(torch.randn((200, 2, 3), generator=gen) * 0.5) / 100.0 * size
    dh = torch.randn((200, 384), generator=gen).double()
    g, u = (R.values(codes[:, i], factors[:, i], R.E4M3, 1) for i in (0, 1))
    if size > 1e6:
        u = u / size
    for fmt in (R.E4M3, R.E5M2):
        for value, bound in B.backward(dh, g, u, act):
            assert B.loose(value, bound, fmt) < 0.01


@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("size", [1e-6, 2.0, 30.0, 1e4])
def test_forward_bounds_are_small(act, size):
    gen = torch.Generator().manual_seed(4)
    m, n, k = 40, 384, 512
    a = R.finite_codes((m, k), R.E4M3, gen, "cpu")
    b = R.finite_codes((2, n, k), R.E4M3, gen, "cpu")
    rms = R.decode_table(R.E4M3)[:0x7F].square().mean().sqrt().item()
    av = R.values(a, torch.exp(torch.randn((m, 4), generator=gen) * 0.5) / rms, R.E4M3, 1)
    g, u = (R.product(av, R.values(b[i], torch.exp(torch.randn((3, 4), generator=gen) * 0.3) / rms * size / math.sqrt(k), R.E4M3, 128))
            for i in (0, 1))
    assert B.loose(*B.gated(g[0], u[0], g[1], u[1], act), R.E4M3) < 0.05
