"""Error bounds of the gated activation's fp32 evaluation that stay far below the values where
the sigmoid saturates, too.

With t = -y log2 e, e = 2^t and s = 1 / (1 + e) (y as in gated_reference):
 - t has at most four roundings (GELU's polynomial: constants, square, sum, product), so e is off
   by |y| 2^-22 of its value, and by two units in the last place, 2^-22, of the exponential;
   ds / s = -(1 - s) de / e, so s by s (1 - s) (|y| + 1) 2^-22.
 - The sum 1 + e and the reciprocal (two units) add (2^-24 + 2^-22) s; but from y = 18 on, e is
   below 2^-25, the sum is 1, and s is 1, off by 1 - s itself.
 - A reciprocal below 2^-126 becomes 0: s is off by itself.
act = g s is off by |g| ds and a rounding.  act' = s + act (1 - s) y' is off by ds, |act| y' ds and
a rounding of 1 - s, (1 - s) y' times act's error, three roundings in y' (GELU: constants, square,
sum) and one of each product, and one of the sum.
For a g known to within eg: act moves by sup |act'| eg, act' by sup |act''| eg.  Both fall with
|g| beyond 4, with act'(g) = 1 - act'(-g): for m = |g| - eg > 4, with tail = |act'(-m)|, |act'| is at most tail (g < 0)
or 1 + tail, and |act''| at most tail (y' + 1).  Elsewhere |act'| < 1.13 and |act''| < 0.8.
"""
from __future__ import annotations

import torch

import gated_reference as G
import gemm_reference as R

ULP = 2.0 ** -24  # half a unit in the last place, of a value
MORE = 1.001      # products of two errors


def _fine(t):
    return t.abs().nan_to_num(0, 0, 0)


def slope_of(g, act):
    y, dy = G.argument(g, act)
    return torch.sigmoid(y) + g * torch.sigmoid(y) * torch.sigmoid(-y) * dy


def activation(g, act, eg):
    """act(g), act'(g) and bounds of their fp32 evaluations for a g known to within eg."""
    y, dy = G.argument(g, act)
    s, rest = torch.sigmoid(y), torch.sigmoid(-y)
    a = g * s
    slope = slope_of(g, act)
    rounds = G.argument(g - eg, act)[0] < 18
    dy = dy.clamp(max=222.0)  # (GELU: from |g| = 32 on the kernel's stays as it is there, 220.8, and s or 1 - s is 0)
    es = s * (rest * (y.abs() + 1) * 2.0 ** -22 + torch.where(rounds, s.new_tensor(2.0 ** -24 + 2.0 ** -22), rest))
    es = es + torch.where(s < 2.0 ** -120, s.clamp(max=2.0 ** -126), 0.0)
    ea = g.abs() * es + ULP * a.abs() + 2.0 ** -149
    product = (a * rest).abs() * dy
    eslope = es + a.abs() * dy * (es + ULP * rest) + dy * rest * ea + 5 * ULP * product + ULP * slope.abs()
    m = g.abs() - eg
    far = m > 4
    tail = slope_of(-m.clamp(min=4), act).abs()
    steep = torch.where(far, torch.where(g < 0, tail, 1 + tail), (slope.abs() + 0.8 * eg).clamp(max=1.13))
    bent = torch.where(far, tail * (G.argument(g.abs() + eg, act)[1] + 1), torch.full_like(g, 0.8))
    return a, slope, _fine(ea * MORE + steep * eg), _fine(eslope * MORE + bent * eg)


def gated(g, u, eg, eu, act):
    """h and its bound, for g and u known to within eg and eu."""
    a, _, ea, _ = activation(g, act, eg)
    return a * u, _fine(a) * eu + ea * _fine(u) + ea * eu + MORE * ULP * _fine(a * u) + 2.0 ** -147


def backward(dh, g, u, act):
    """(value, bound) of dg, du and h, for codes' values g and u (fp32: one rounding each)."""
    a, slope, ea, es = activation(g, act, ULP * _fine(g))
    # (fp32 products that leave the normal range are off by up to 2^-149 each)
    return ((dh * u * slope, _fine(dh * u) * (es + 4 * ULP * _fine(slope)) * MORE + 2.0 ** -147),
            (dh * a, _fine(dh) * (ea + 2 * ULP * _fine(a)) * MORE + 2.0 ** -147),
            (a * u, _fine(u) * (ea + 3 * ULP * _fine(a)) * MORE + 2.0 ** -147))


def loose(value, bound, fmt):
    """The share of elements whose bound a code's error does not hide: neither below a sixteenth of
    the value nor below a thousandth of the smallest code of its 1 x 128 tile."""
    step = G.tile_max(_fine(value)).repeat_interleave(128, -1)[..., :value.shape[-1]] / G.TOP[fmt] * G.LEAST[fmt]
    return float(((bound > value.abs() / 16) & (bound > step / 1024)).double().mean())


def check_forward(outs, gu, bound, act):
    """Outputs (h, factors, optionally both projections and factors) against projections gu [m, 2, n]."""
    h, eh = gated(gu[:, 0], gu[:, 1], bound[:, 0], bound[:, 1], act)
    G.check_tiles(outs[0], outs[1], h, eh, R.E4M3)
    if len(outs) > 2:
        G.check_tiles(outs[2], outs[3], gu, bound, R.E4M3)


def check_backward(outs, dh, gu, sgu, act, fmt):
    """The six outputs (None: left out) against dh and the checkpoint."""
    g, u = (R.values(gu[:, i], sgu[:, i], R.E4M3, 1) for i in (0, 1))
    parts = backward(dh.double(), g, u, act)
    for i in (0, 1):
        if outs[0] is not None:
            G.check_tiles(outs[0][:, i], outs[1][:, i], *parts[i], fmt)
        if outs[2] is not None:
            G.check_tiles(outs[2][i], outs[3][i], parts[i][0].T, parts[i][1].T, fmt)
    if outs[4] is not None:
        G.check_tiles(outs[4], outs[5], parts[2][0].T, parts[2][1].T, R.E4M3)
