"""Plain 64-bit reference of the block-scaled FP8 products, and its error bound.

A product's fp32 evaluation adds 128 exact products per block, multiplies by
the block's scale and adds the blocks.  With every addition correct to 2^-23
(fp32 rounding, or the truncating alignment of a tensor core) and the two
scale products to 2^-24, the error of an output is at most
    (128 + blocks + 4) * 2^-23 * sum_k |A[i, k] B[j, k]|
and a BF16 result lies between the roundings of the two ends of that interval
(rounding is monotone).
"""
from __future__ import annotations

import math

import torch

E4M3, E5M2 = 0, 1


def decode_table(fmt: int) -> torch.Tensor:
    e_bits, bias = (4, 7) if fmt == E4M3 else (5, 15)
    m_bits = 7 - e_bits
    out = []
    for code in range(256):
        e, f = (code >> m_bits) & ((1 << e_bits) - 1), code & ((1 << m_bits) - 1)
        v = math.ldexp(1 + f / 2 ** m_bits, e - bias) if e else math.ldexp(f / 2 ** m_bits, 1 - bias)
        if fmt == E4M3 and e == 15 and f == 7:
            v = math.nan
        elif fmt == E5M2 and e == 31:
            v = math.nan if f else math.inf
        out.append(-v if code & 0x80 else v)
    return torch.tensor(out, dtype=torch.float64)


def values(q, scale_inv, fmt, block_rows):
    """Dequantized [rows, cols] in 64 bits (scales indexed by row block and 128-column block)."""
    rows, cols = q.shape
    r = torch.arange(rows, device=q.device)[:, None] // block_rows
    c = torch.arange(cols, device=q.device)[None, :] // 128
    return decode_table(fmt).to(q.device)[q.long()] * scale_inv.double()[r, c]


def finite_codes(shape, fmt, gen, device):
    """Random codes over the whole finite range of the format."""
    top = 0x7E if fmt == E4M3 else 0x7B
    mag = torch.randint(0, top + 1, shape, generator=gen, device=device, dtype=torch.int64)
    sign = torch.randint(0, 2, shape, generator=gen, device=device, dtype=torch.int64)
    return (mag | (sign << 7)).to(torch.uint8)


def scales(shape, gen, device):
    return torch.exp(torch.randn(shape, generator=gen, device=device) * 2 - 3)


def product(av, bv):
    """(value, bound on the fp32 evaluation's error) of av [m, k] times bv [n, k]^T."""
    blocks = -(-av.shape[1] // 128) if av.shape[1] else 0
    gamma = (128 + blocks + 4) * 2.0 ** -23
    return av @ bv.T, gamma * (av.abs().nan_to_num(0, 0, 0) @ bv.abs().nan_to_num(0, 0, 0).T)


def check(d, want, bound):
    """d within [want - bound, want + bound] rounded to its type; NaN and Inf where want has them."""
    got = d.double()
    assert torch.equal(got.isnan(), want.isnan()), "NaN at other places"
    inf = want.isinf()
    assert torch.equal(got.isinf(), inf) and torch.equal(got[inf], want[inf]), "Inf at other places"
    fine = want.isfinite()
    got, want, bound = got[fine], want[fine], bound[fine]
    lo, hi = ((want + sign * (bound + 1e-37)) for sign in (-1, 1))
    if d.dtype == torch.bfloat16:
        lo, hi = lo.bfloat16().double(), hi.bfloat16().double()
    bad = (got < lo) | (got > hi)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst {((got - want).abs() / bound).max():.3g} bounds"
