"""Global gradient norm and clipping on the GPU against 64 bits.

A thread adds at most 16 * reps squares per fp32 sum (reps: chunks of 32 KB
per CTA, more than one above 8192 of them), so the sum of squares is right to
(16 * reps + 2) * 2^-24 and the norm, its rounding included, to (16 * reps + 4)
* 2^-24; the factor adds two roundings and the product one.
"""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def make(sizes, dtypes, seed=0, std=1e-2):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device=DEV) * std).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


def norm64(xs):
    return sum(((x.double() ** 2).sum() for x in xs), torch.zeros((), dtype=torch.float64, device=DEV)).sqrt()


def norm_bound(xs):
    chunks = sum(-(-x.numel() * x.element_size() // 32768) for x in xs)
    reps = 1 if chunks <= 8192 else -(-chunks // (8192 - len(xs)))
    return (16 * reps + 4) * 2.0 ** -24


def check(xs, ys, max_norm, norm, coef, eps=1e-6):
    want, rel = norm64(xs), norm_bound(xs)
    assert abs(norm.double() - want) <= rel * want
    factor = min(1.0, max_norm / (float(want) + eps)) if want + eps > 0 else 1.0
    rel += 2 * 2.0 ** -24
    assert abs(float(coef) - factor) <= rel * factor
    for x, y in zip(xs, ys):
        v = x.double() * factor
        e = v.abs() * (rel + 2.0 ** -24) + 2.0 ** -149
        lo, hi = (v - e).to(y.dtype).double(), (v + e).to(y.dtype).double()
        assert ((y.double() >= lo) & (y.double() <= hi)).all()


def clip(xs, max_norm, ys=None, **kw):
    norm, coef = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    fq.fp8_grad_clip_grouped(xs, max_norm, norm, ys=ys, coef_out=coef, **kw)
    return norm, coef


SIZES = {
    "one": [1], "few": [7, 8, 9, 15, 16, 17], "empty": [0, 5, 0], "vector": [4096], "chunk": [16384], "chunks": [16383, 16385, 8191, 8193],
    "matrix": [1024 * 1000], "mixed": [3, 100000, 1, 77777, 2048, 0, 31], "many": [(37 * i) % 1000 for i in range(300)],
    "thousands": [1 + (i % 5) for i in range(2500)], "matrices": [3_000_000, 4_000_001, 5_000_000],
}


@pytest.mark.parametrize("out", [None, BF16, F32])
@pytest.mark.parametrize("dtypes", [[BF16], [F32], [BF16, BF16, F32]])
@pytest.mark.parametrize("kind", list(SIZES))
def test_clip(kind, dtypes, out):
    xs = make(SIZES[kind], dtypes, 3)
    before = [x.clone() for x in xs]
    want = norm64(xs)
    for max_norm in (float(want) * 0.3, float(want) * 2 + 1):
        ys = None if out is None else [torch.full(x.shape, 9.0, dtype=out, device=DEV) for x in xs]
        norm, coef = clip(xs, max_norm, ys)
        check(before, xs if ys is None else ys, max_norm, norm, coef)
        if ys is None:
            for x, b in zip(xs, before):
                x.copy_(b)
        else:
            assert all(torch.equal(x, b) for x, b in zip(xs, before))


@pytest.mark.parametrize("kind", list(SIZES))
def test_norm_alone(kind):
    xs = make(SIZES[kind], [BF16, F32], 5)
    norm = torch.empty(1, device=DEV)
    fq.fp8_grad_norm_grouped(xs, norm)
    want = norm64(xs)
    assert abs(norm.double() - want) <= norm_bound(xs) * want
    again = torch.empty(1, device=DEV)
    fq.fp8_grad_norm_grouped(xs, again)
    assert torch.equal(norm, again)


def test_in_place_without_clipping_writes_nothing():
    xs = make([100001, 33], [BF16])
    before = [x.clone() for x in xs]
    _, coef = clip(xs, 1e9)
    assert coef.item() == 1.0 and all(torch.equal(x, b) for x, b in zip(xs, before))


@pytest.mark.parametrize("shift_x,shift_y", [(1, 0), (0, 1), (1, 3), (4, 4), (8, 8)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_views_and_canaries(dtype, out, shift_x, shift_y):
    n = 40001
    flat = make([n + 64], [dtype], 7)[0]
    buf = torch.full((n + 64,), 55.0, dtype=out, device=DEV)
    x, y = flat[shift_x:shift_x + n], buf[shift_y:shift_y + n]
    norm, coef = clip([x], 0.25, [y])
    check([x], [y], 0.25, norm, coef)
    assert (buf[:shift_y] == 55.0).all() and (buf[shift_y + n:] == 55.0).all()


@pytest.mark.parametrize("std", [1e-38, 1e-30, 1e-22, 1e-16, 1e16, 1e22, 1e30])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_squares_outside_the_fp32_range(dtype, std):
    xs = make([20000, 333], [dtype], 2, std)
    norm = torch.empty(1, device=DEV)
    fq.fp8_grad_norm_grouped(xs, norm)
    want = norm64(xs)
    assert abs(norm.double() - want) <= norm_bound(xs) * want + 2.0 ** -149


def test_large_and_small_tensors_together():
    xs = make([50000], [F32], 1, 1e25) + make([50000], [F32], 2, 1e-25) + [torch.zeros(70000, device=DEV)]
    norm, coef = clip(xs, 1.0, [torch.empty_like(x) for x in xs])
    want = norm64(xs)
    assert abs(norm.double() - want) <= norm_bound(xs) * want


@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_not_finite(dtype, bad):
    xs = make([40000, 100], [dtype], 1)
    xs[1][37] = bad
    ys = [torch.empty(x.shape, dtype=F32, device=DEV) for x in xs]
    norm, coef = clip(xs, 0.1, ys)
    assert not norm.isfinite().item() and (norm.isnan().item() == (bad != bad)) and coef.item() == 1.0
    for x, y in zip(xs, ys):
        assert torch.equal(y.nan_to_num(7.0), x.float().nan_to_num(7.0))


def test_norm_beyond_fp32_is_inf_and_clips_nothing():
    xs = [torch.full((100,), 3e38, device=DEV)]
    norm, coef = clip(xs, 1.0)
    assert norm.item() == INF and coef.item() == 1.0 and (xs[0] == 3e38).all()


def test_all_zero_and_zero_max_norm():
    xs = [torch.zeros(5000, device=DEV), torch.zeros(33, dtype=BF16, device=DEV)]
    norm, coef = clip(xs, 0.5)
    assert norm.item() == 0.0 and coef.item() == 1.0
    xs = make([1000], [F32])
    norm, coef = clip(xs, 0.0)
    assert coef.item() == 0.0 and (xs[0] == 0).all()


def test_more_than_the_partial_slots():
    """1.2 GB: more chunks than partial slots, so a CTA takes several chunks."""
    xs = make([300_000_000, 100, 299_999_999], [BF16], 4)
    ys = [torch.empty_like(x) for x in xs]
    norm, coef = clip(xs, 1.0, ys)
    check(xs, ys, 1.0, norm, coef)


def test_other_stream_and_graph():
    xs = make([100000, 77], [BF16, F32], 6)
    ys = [torch.empty_like(x) for x in xs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    norm, coef = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    fq.fp8_grad_clip_grouped(xs, 0.1, norm, ys=ys, coef_out=coef, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check(xs, ys, 0.1, norm, coef)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fq.fp8_grad_clip_grouped(xs, 0.1, norm, ys=ys, coef_out=coef)
    for y in ys:
        y.zero_()
    xs[0].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    check(xs, ys, 0.1, norm, coef)
