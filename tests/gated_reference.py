"""Plain 64-bit reference of the gated feed-forward block, with bounds of its fp32 evaluation.

act(g) = g s, s = sigmoid(y); y = g (SiLU) or 2 c (g + 0.044715 g^3) (GELU, tanh form).
In fp32 the sigmoid's exponential is off by (|y| + 4) 2^-22 of its value (the argument,
three roundings of it at most; two units in the last place each of the exponential and the
reciprocal), so act(g) by (|y| + 8) 2^-22 of its value with the products around it, and
act'(g) = s + act(g) (1 - s) y' by (|y| + 8) 2^-22 (1 + |g| y'); |act'| < 1.2.  What is below
1e-36 may be 0.  A code is off by half a step of its value: 2^-4 (E4M3) or 2^-3 (E5M2) of
it, or half the smallest value.
"""
from __future__ import annotations

import math

import torch

import gemm_reference as R

SILU, GELU = 0, 1
TOP = {R.E4M3: 448.0, R.E5M2: 57344.0}
HALF = {R.E4M3: 2.0 ** -4, R.E5M2: 2.0 ** -3}
LEAST = {R.E4M3: 2.0 ** -9, R.E5M2: 2.0 ** -16}


def blocks(n):
    return -(-n // 128)


def argument(g, act):
    """y and y'."""
    if act == SILU:
        return g, torch.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)


def activation(g, act):
    """act(g), act'(g) and the bounds of their fp32 evaluations."""
    y, dy = argument(g, act)
    s, rest = torch.sigmoid(y), torch.sigmoid(-y)
    a = g * s
    slope = s + a * rest * dy
    far = (y.abs().nan_to_num(0, 0, 0) + 8) * 2.0 ** -22
    far_slope = far * (1 + (g * dy).abs().nan_to_num(0, 0, 0)).clamp(max=1e6)
    return a, slope, far * a.abs().nan_to_num(0, 0, 0) + 1e-36, far_slope


def gated(g, u, eg, eu, act):
    """h and its bound, for g and u known to within eg and eu."""
    a, _, ea, _ = activation(g, act)
    ea = ea + 1.2 * eg
    fine = lambda t: t.abs().nan_to_num(0, 0, 0)  # noqa: E731
    return a * u, fine(a) * eu + ea * fine(u) + ea * eu + fine(a * u) * 2.0 ** -22


def backward(dh, g, u, act):
    """(value, bound) of dg, du and h, for codes' values g and u (fp32 factors: one rounding)."""
    a, slope, ea, es = activation(g, act)
    fine = lambda t: t.abs().nan_to_num(0, 0, 0)  # noqa: E731
    ea, es = ea + 1.2 * fine(g) * 2.0 ** -23, es + fine(g) * 2.0 ** -22
    tiny = 2.0 ** -22
    # (fp32 products that leave the normal range are off by up to 2^-149 each)
    return ((dh * u * slope, fine(dh * u) * (es + tiny * (fine(slope) + 1)) + 2.0 ** -147),
            (dh * a, fine(dh) * (ea + tiny * fine(a)) + 2.0 ** -147), (a * u, fine(u) * (ea + tiny * fine(a)) + 2.0 ** -147))


def tile_max(v):
    """[r, c] -> [r, blocks of c]: the largest of each 1 x 128 tile."""
    return torch.stack([p.amax(-1) for p in v.split(128, -1)], -1)


def check_tiles(q, inv, value, bound, fmt):
    """Codes q and factors inv of 1 x 128 tiles along the last axis against values known to within bound."""
    assert q.shape == value.shape and inv.shape == (*value.shape[:-1], blocks(value.shape[-1]))
    top = TOP[fmt]
    wide = lambda t: t.repeat_interleave(128, -1)[..., :value.shape[-1]]  # noqa: E731
    special = tile_max((~value.isfinite()).double()) > 0
    amax, most = tile_max(value.abs().nan_to_num(0, 0, 0)), tile_max(bound)
    inv = inv.double()
    plain = special | (amax == 0)
    assert (inv[plain] == 1).all(), "factor of a tile of zeros, or with Inf or NaN"
    want = amax / top
    # A tile whose largest value is not beyond its bound (act(g) below 1e-36) may be one of
    # zeros to the kernel, and that has factor 1.
    zeros = (amax <= most) & (inv == 1)
    off = ((inv - want).abs() > most / top + 4 * 2.0 ** -24 * want + 1e-38) & ~plain & ~zeros
    assert not off.any(), f"{int(off.sum())} of {off.numel()} factors: {inv[off][:3].tolist()} for {want[off][:3].tolist()}"
    got = R.decode_table(fmt).to(q.device)[q.long()] * wide(inv)
    assert torch.equal(got.isnan(), value.isnan()), "NaN at other places"
    inf = value.isinf()
    end = math.inf if fmt == R.E5M2 else top
    assert torch.equal(got[inf], value[inf].sign() * end), "Inf"
    fine = value.isfinite()
    limit = top * wide(inv)
    near = torch.minimum(torch.maximum(value, -limit), limit)[fine]
    got, e, v, f = got[fine], bound[fine], value[fine].abs(), wide(inv)[fine]
    allowed = e + torch.maximum(HALF[fmt] * (v + e) * (1 + 2.0 ** -20), f * LEAST[fmt] / 2 * (1 + 2.0 ** -20))
    bad = (got - near).abs() > allowed
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes, worst {float(((got - near).abs() / allowed).max()):.4g} of what is allowed"
