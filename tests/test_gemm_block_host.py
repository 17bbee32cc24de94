"""Refusals of the block-scaled products and of gradient clipping: checked on the host, nothing launched."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq

BAD = 0x1000  # never dereferenced


def gemm(L, fmt_a=0, fmt_b=0, layout=0, rows=128, m=4, n=4, k=4, a=BAD, sa=BAD, b=BAD, sb=BAD, d=BAD, out=0, acc=0):
    return L.fp8_gemm_block(a, fmt_a, sa, b, fmt_b, sb, layout, rows, m, n, k, d, out, acc, None)


def grouped(L, groups=2, ends=BAD, fmt_a=0, layout=0, rows=4, n=4, k=4, a=BAD, sb=BAD, d=BAD, out=0):
    return L.fp8_gemm_block_grouped(groups, ends, a, fmt_a, BAD, BAD, 0, sb, layout, rows, n, k, d, out, None)


def wgrad(L, groups=2, ends=BAD, m=4, n=4, rows=4, d=BAD, out=1, acc=0, fmt_b=0):
    return L.fp8_gemm_block_grouped_wgrad(groups, ends, BAD, 0, BAD, BAD, fmt_b, BAD, m, n, rows, d, out, acc, None)


@pytest.mark.parametrize("call,status,msg", [
    (lambda L: gemm(L, fmt_a=2), 1, "unknown format"),
    (lambda L: gemm(L, fmt_b=-1), 1, "unknown format"),
    (lambda L: gemm(L, out=3), 1, "out_dtype"),
    (lambda L: gemm(L, layout=2), 1, "layout"),
    (lambda L: gemm(L, m=-1), 1, "negative size"),
    (lambda L: gemm(L, k=-1), 1, "negative size"),
    (lambda L: gemm(L, rows=64), 2, "b_block_rows"),
    (lambda L: gemm(L, rows=1, layout=1), 2, "along the contraction"),
    (lambda L: gemm(L, acc=1, out=0), 2, "accumulate"),
    (lambda L: gemm(L, m=2 ** 31), 2, "below 2^31"),
    (lambda L: gemm(L, m=2 ** 30, n=2 ** 30), 2, "too many output tiles"),
    (lambda L: gemm(L, d=None), 1, "d is NULL"),
    (lambda L: gemm(L, d=BAD + 1), 1, "element-aligned"),
    (lambda L: gemm(L, d=BAD + 2, out=1), 1, "element-aligned"),
    (lambda L: gemm(L, a=None), 1, "NULL"),
    (lambda L: gemm(L, b=None), 1, "NULL"),
    (lambda L: gemm(L, sa=None), 1, "NULL"),
    (lambda L: gemm(L, sb=BAD + 2), 1, "4-byte aligned"),
    (lambda L: grouped(L, groups=0), 1, "groups must be"),
    (lambda L: grouped(L, groups=1025), 1, "groups must be"),
    (lambda L: grouped(L, ends=None), 1, "group_ends is NULL"),
    (lambda L: grouped(L, ends=BAD + 4), 1, "8-byte aligned"),
    (lambda L: grouped(L, rows=-1), 1, "negative size"),
    (lambda L: grouped(L, d=None), 1, "d is NULL"),
    (lambda L: grouped(L, a=None), 1, "NULL"),
    (lambda L: grouped(L, sb=None), 1, "NULL"),
    (lambda L: grouped(L, layout=7), 1, "layout"),
    (lambda L: wgrad(L, groups=-3), 1, "groups must be"),
    (lambda L: wgrad(L, ends=None), 1, "group_ends is NULL"),
    (lambda L: wgrad(L, fmt_b=9), 1, "unknown format"),
    (lambda L: wgrad(L, out=0, acc=1), 2, "accumulate"),
    (lambda L: wgrad(L, n=-1), 1, "negative size"),
    (lambda L: wgrad(L, groups=1024, m=2 ** 20, n=2 ** 20), 2, "too many output tiles"),
])
def test_products_refuse_before_launch(native_lib, call, status, msg):
    before = native_lib.fp8_launch_count()
    assert call(native_lib) == status
    assert msg in native_lib.fp8_last_error_message().decode()
    assert native_lib.fp8_launch_count() == before


def test_empty_products_need_no_device(native_lib):
    assert gemm(native_lib, m=0, a=None, b=None, sa=None, sb=None, d=None) == 0
    assert gemm(native_lib, n=0, d=None) == 0
    assert gemm(native_lib, k=0, acc=1, out=1, a=None, b=None, sa=None, sb=None) == 0
    assert grouped(native_lib, rows=0, a=None, d=None) == 0
    assert wgrad(native_lib, m=0, d=None) == 0


def _u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


@pytest.mark.parametrize("kw,msg", [
    (dict(a=torch.zeros(4, 256)), "a must be uint8"),
    (dict(a=_u8(4, 256, 1)), "2-D"),
    (dict(sa=torch.zeros(4, 3)), "scale_inv_a"),
    (dict(sa=torch.zeros(4, 2, dtype=torch.float64)), "scale_inv_a"),
    (dict(b=_u8(130, 255)), "b must be uint8"),
    (dict(b=_u8(256, 130)), "b must be uint8"),
    (dict(sb=torch.zeros(130, 2)), "scale_inv_b"),
    (dict(d=torch.zeros(5, 130)), "d must be"),
    (dict(d=torch.zeros(4 * 130)), "d must be"),
    (dict(b_layout=fq.B_KN), "b must be uint8"),
    (dict(b_block_rows=1), "scale_inv_b"),
    (dict(), "CUDA device"),
])
def test_binding_checks_shapes(native_lib, kw, msg):
    args = dict(a=_u8(4, 256), sa=torch.zeros(4, 2), b=_u8(130, 256), sb=torch.zeros(2, 2), d=torch.zeros(4, 130))
    extra = {k: kw.pop(k) for k in ("b_layout", "b_block_rows") if k in kw}
    args.update(kw)
    with pytest.raises(ValueError, match=msg):
        fq.fp8_gemm_block(args["a"], args["sa"], args["b"], args["sb"], args["d"], **extra)


def test_grouped_bindings_check_shapes(native_lib):
    a, sa, b, sb, d = _u8(6, 256), torch.zeros(6, 2), _u8(3, 130, 256), torch.zeros(3, 2, 2), torch.zeros(6, 130)
    ends = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="group_ends"):
        fq.fp8_gemm_block_grouped(a, sa, b, sb, ends.int(), d)
    with pytest.raises(ValueError, match="b must be uint8"):
        fq.fp8_gemm_block_grouped(a, sa, b, sb, ends[:2].clone(), d)
    with pytest.raises(ValueError, match="d must be"):
        fq.fp8_gemm_block_grouped(a, sa, b, sb, ends, d[:5])
    with pytest.raises(ValueError, match="CUDA device"):
        fq.fp8_gemm_block_grouped(a, sa, b, sb, ends, d)
    at, st, bt, tt = _u8(130, 6), torch.zeros(130, 1), _u8(256, 6), torch.zeros(256, 1)
    with pytest.raises(ValueError, match="d must be"):
        fq.fp8_gemm_block_grouped_wgrad(at, st, bt, tt, ends, torch.zeros(2, 130, 256))
    with pytest.raises(ValueError, match="b must be uint8"):
        fq.fp8_gemm_block_grouped_wgrad(at, st, _u8(256, 7), tt, ends, torch.zeros(3, 130, 256))
    with pytest.raises(ValueError, match="CUDA device"):
        fq.fp8_gemm_block_grouped_wgrad(at, st, bt, tt, ends, torch.zeros(3, 130, 256))


# ------------------------------------------------------------ gradient clipping

def _arr(kind, vals):
    from array import array
    return array(kind, vals)


def clip(L, count=1, xs=(BAD,), ns=(4,), dt=(0,), ys=None, yd=None, max_norm=1.0, eps=1e-6, norm=BAD, coef=None, norm_only=False):
    a = [_arr(k, v) if v is not None else None for k, v in (("Q", xs), ("q", ns), ("i", dt), ("Q", ys), ("i", yd))]
    p = [v.buffer_info()[0] if v is not None else None for v in a]
    if norm_only:
        return L.fp8_grad_norm_grouped(count, p[0], p[1], p[2], norm, None)
    return L.fp8_grad_clip_grouped(count, *p, max_norm, eps, norm, coef, None)


@pytest.mark.parametrize("call,status,msg", [
    (lambda L: clip(L, count=0), 1, "count must be"),
    (lambda L: clip(L, count=4097), 1, "count must be"),
    (lambda L: clip(L, xs=None), 1, "is NULL"),
    (lambda L: clip(L, ns=(-1,)), 1, "n < 0"),
    (lambda L: clip(L, dt=(5,)), 1, "unknown dtype"),
    (lambda L: clip(L, xs=(0,)), 1, "tensor 0 is NULL"),
    (lambda L: clip(L, xs=(BAD + 1,)), 1, "element-aligned"),
    (lambda L: clip(L, ys=(BAD,)), 1, "both"),
    (lambda L: clip(L, ys=(BAD,), yd=(7,)), 1, "unknown dtype"),
    (lambda L: clip(L, ys=(0,), yd=(0,)), 1, "output 0 is NULL"),
    (lambda L: clip(L, ys=(BAD + 2,), yd=(1,)), 1, "element-aligned"),
    (lambda L: clip(L, ys=(BAD,), yd=(1,)), 2, "another type"),
    (lambda L: clip(L, max_norm=-1.0), 1, "max_norm"),
    (lambda L: clip(L, max_norm=float("nan")), 1, "max_norm"),
    (lambda L: clip(L, max_norm=float("inf")), 1, "max_norm"),
    (lambda L: clip(L, eps=-1.0), 1, "eps"),
    (lambda L: clip(L, norm=BAD + 2), 1, "4-byte aligned"),
    (lambda L: clip(L, norm=None, norm_only=True), 1, "norm_out is NULL"),
    (lambda L: clip(L, count=4097, norm_only=True), 1, "count must be"),
])
def test_clip_refuses_before_launch(native_lib, call, status, msg):
    before = native_lib.fp8_launch_count()
    assert call(native_lib) == status
    assert msg in native_lib.fp8_last_error_message().decode()
    assert native_lib.fp8_launch_count() == before


def test_clip_binding_checks(native_lib):
    xs = [torch.zeros(8), torch.zeros(4, dtype=torch.bfloat16)]
    with pytest.raises(ValueError, match="CUDA device"):
        fq.fp8_grad_clip_grouped(xs, 1.0)
    with pytest.raises(ValueError, match="non-empty"):
        fq.fp8_grad_clip_grouped([], 1.0)
    with pytest.raises(ValueError, match="as long as"):
        fq.fp8_grad_clip_grouped(xs, 1.0, ys=xs[:1])
    with pytest.raises(ValueError, match="as many elements"):
        fq.fp8_grad_clip_grouped(xs, 1.0, ys=xs[::-1])
    with pytest.raises(ValueError, match="non-empty"):
        fq.fp8_grad_norm_grouped([], torch.zeros(1))


# ------------------------------------------------------------ a layer's step

def test_block_linear_step_refuses_and_accounts():
    from fp8_scaled_quantization_gb300 import pipelines as P
    meta = torch.device("meta")
    mk = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=meta)  # noqa: E731
    with pytest.raises(ValueError, match="group_ends"):
        P.BlockLinearStep(mk(8, 256), mk(2, 128, 256), mk(8, 128))
    with pytest.raises(ValueError, match="multiple of 128"):
        P.BlockLinearStep(mk(8, 256), mk(2, 100, 256), mk(8, 100), torch.empty(2, dtype=torch.int64, device=meta))
    b = P.BlockLinearStep(mk(512, 256), mk(128, 256), mk(512, 128)).bytes()
    codes, tokens = 128 * 256, 512
    assert b.per_kernel["forward"] == (tokens * 256 + 4 * tokens * 2 + codes + 4 * 2 + tokens * 128 * 2, 1)
    assert b.per_kernel["dgrad"] == (tokens * 128 + 4 * tokens + codes + 4 * 2 + tokens * 256 * 2, 1)
    assert b.per_kernel["wgrad"] == (tokens * 384 + 4 * 384 * 4 + codes * 4, 1)
    assert b.per_kernel["clip"] == (codes * 8, 1) and b.launches == 7
