"""The gated feed-forward block: refusals on the host (nothing launched), and the 64-bit
reference itself against differences."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gated_reference as G

BAD = 0x1000  # never dereferenced


def gated(L, fmt_a=0, fmt_b=0, act=0, m=4, n=4, k=4, a=BAD, sa=BAD, b=BAD, sb=BAD, h=BAD, sh=BAD, gu=None, sgu=None):
    return L.fp8_gemm_block_gated(a, fmt_a, sa, b, fmt_b, sb, act, m, n, k, h, sh, gu, sgu, None)


def grouped(L, groups=2, ends=BAD, act=0, rows=4, n=4, k=4, b=BAD, h=BAD, sh=BAD, gu=None, sgu=None):
    return L.fp8_gemm_block_gated_grouped(groups, ends, BAD, 0, BAD, b, 0, BAD, act, rows, n, k, h, sh, gu, sgu, None)


def backward(L, dt=0, act=0, rows=4, n=4, fmt=0, dh=BAD, gu=BAD, sgu=BAD, dgu=BAD, sdgu=BAD, dt_=BAD, sdt=BAD, ht=BAD,
             sht=BAD):
    return L.fp8_gated_block_backward(dh, dt, gu, sgu, act, rows, n, fmt, dgu, sdgu, dt_, sdt, ht, sht, None)


@pytest.mark.parametrize("call,status,msg", [
    (lambda L: gated(L, fmt_a=2), 1, "unknown format"),
    (lambda L: gated(L, fmt_b=-1), 1, "unknown format"),
    (lambda L: gated(L, act=2), 1, "unknown activation"),
    (lambda L: gated(L, act=-1), 1, "unknown activation"),
    (lambda L: gated(L, m=-1), 1, "negative size"),
    (lambda L: gated(L, n=-1), 1, "negative size"),
    (lambda L: gated(L, k=-1), 1, "negative size"),
    (lambda L: gated(L, k=2 ** 31), 2, "below 2^31"),
    (lambda L: gated(L, m=2 ** 21, n=2 ** 21), 2, "too many output tiles"),
    (lambda L: gated(L, gu=BAD), 1, "both"),
    (lambda L: gated(L, sgu=BAD), 1, "both"),
    (lambda L: gated(L, h=None), 1, "h or its scales"),
    (lambda L: gated(L, sh=None), 1, "h or its scales"),
    (lambda L: gated(L, a=None), 1, "an operand"),
    (lambda L: gated(L, sb=None), 1, "an operand"),
    (lambda L: gated(L, sa=BAD + 2), 1, "4-byte aligned"),
    (lambda L: gated(L, sh=BAD + 1), 1, "4-byte aligned"),
    (lambda L: gated(L, gu=BAD, sgu=BAD + 2), 1, "4-byte aligned"),
    (lambda L: grouped(L, groups=0), 1, "groups must be"),
    (lambda L: grouped(L, groups=1025), 1, "groups must be"),
    (lambda L: grouped(L, ends=None), 1, "group_ends is NULL"),
    (lambda L: grouped(L, ends=BAD + 4), 1, "8-byte aligned"),
    (lambda L: grouped(L, act=5), 1, "unknown activation"),
    (lambda L: grouped(L, rows=-1), 1, "negative size"),
    (lambda L: grouped(L, b=None), 1, "an operand"),
    (lambda L: grouped(L, h=None), 1, "h or its scales"),
    (lambda L: grouped(L, gu=BAD), 1, "both"),
    (lambda L: grouped(L, groups=1024, rows=2 ** 30, n=2 ** 14), 2, "too many output tiles"),
    (lambda L: backward(L, dt=2), 1, "unknown dtype"),
    (lambda L: backward(L, fmt=2), 1, "unknown format"),
    (lambda L: backward(L, act=2), 1, "unknown activation"),
    (lambda L: backward(L, rows=-1), 1, "negative size"),
    (lambda L: backward(L, n=2 ** 31), 2, "below 2^31"),
    (lambda L: backward(L, rows=2 ** 24, n=2 ** 24), 2, "too many tiles"),
    (lambda L: backward(L, sdgu=None), 1, "both"),
    (lambda L: backward(L, dt_=None), 1, "both"),
    (lambda L: backward(L, sht=None), 1, "both"),
    (lambda L: backward(L, dgu=None, sdgu=None, dt_=None, sdt=None, ht=None, sht=None), 1, "no output"),
    (lambda L: backward(L, dh=None), 1, "an input is NULL"),
    (lambda L: backward(L, gu=None), 1, "an input is NULL"),
    (lambda L: backward(L, sgu=None), 1, "an input is NULL"),
    (lambda L: backward(L, dh=BAD + 1), 1, "element-aligned"),
    (lambda L: backward(L, dt=1, dh=BAD + 2), 1, "element-aligned"),
    (lambda L: backward(L, sgu=BAD + 2), 1, "4-byte aligned"),
    (lambda L: backward(L, sdt=BAD + 2), 1, "4-byte aligned"),
])
def test_refused_before_launch(native_lib, call, status, msg):
    before = native_lib.fp8_launch_count()
    assert call(native_lib) == status
    assert msg in native_lib.fp8_last_error_message().decode()
    assert native_lib.fp8_launch_count() == before


def test_empty_calls_need_no_device(native_lib):
    assert gated(native_lib, m=0, a=None, b=None, sa=None, sb=None, h=None, sh=None) == 0
    assert gated(native_lib, n=0, h=None, sh=None) == 0
    assert grouped(native_lib, rows=0, h=None, sh=None) == 0
    assert backward(native_lib, rows=0, dh=None, gu=None, sgu=None) == 0
    assert backward(native_lib, n=0, dh=None) == 0


def _u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


@pytest.mark.parametrize("kw,msg", [
    (dict(a=torch.zeros(4, 256)), "a must be uint8"),
    (dict(sa=torch.zeros(4, 3)), "scale_inv_a"),
    (dict(b=_u8(130, 256)), "b must be uint8"),
    (dict(b=_u8(260, 256)), "b must be uint8"),
    (dict(sb=torch.zeros(3, 2)), "scale_inv_b"),
    (dict(h=_u8(5, 130)), "h must be"),
    (dict(h=torch.zeros(4, 130)), "h must be uint8"),
    (dict(sh=torch.zeros(4, 1)), "scale_inv_h"),
    (dict(gu=_u8(4, 2, 130)), "go together"),
    (dict(sgu=torch.zeros(4, 2, 2)), "go together"),
    (dict(gu=_u8(4, 260), sgu=torch.zeros(4, 2, 2)), "gu must be uint8"),
    (dict(gu=_u8(4, 2, 130), sgu=torch.zeros(4, 4)), "scale_inv_gu"),
    (dict(), "CUDA device"),
])
def test_binding_checks_shapes(native_lib, kw, msg):
    args = dict(a=_u8(4, 256), sa=torch.zeros(4, 2), b=_u8(2, 130, 256), sb=torch.zeros(2, 2, 2), h=_u8(4, 130),
                sh=torch.zeros(4, 2), gu=None, sgu=None)
    args.update(kw)
    with pytest.raises(ValueError, match=msg):
        fq.fp8_gemm_block_gated(*args.values())


def test_grouped_and_backward_bindings_check_shapes(native_lib):
    a, sa, b, sb = _u8(6, 256), torch.zeros(6, 2), _u8(3, 2, 130, 256), torch.zeros(3, 2, 2, 2)
    h, sh, ends = _u8(6, 130), torch.zeros(6, 2), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="group_ends"):
        fq.fp8_gemm_block_gated_grouped(a, sa, b, sb, ends.int(), h, sh)
    with pytest.raises(ValueError, match="b must be uint8"):
        fq.fp8_gemm_block_gated_grouped(a, sa, b, sb, ends[:2].clone(), h, sh)
    with pytest.raises(ValueError, match="CUDA device"):
        fq.fp8_gemm_block_gated_grouped(a, sa, b, sb, ends, h, sh)
    dh, gu, sgu = torch.zeros(6, 130), _u8(6, 2, 130), torch.zeros(6, 2, 2)
    with pytest.raises(ValueError, match="gu must be uint8"):
        fq.fp8_gated_block_backward(dh, _u8(6, 260), sgu, gu, sgu)
    with pytest.raises(ValueError, match="dgu_t must be uint8"):
        fq.fp8_gated_block_backward(dh, gu, sgu, dgu_t=gu, scale_inv_dgu_t=sgu)
    with pytest.raises(ValueError, match="go together"):
        fq.fp8_gated_block_backward(dh, gu, sgu, h_t=_u8(130, 6))
    with pytest.raises(ValueError, match="CUDA device"):
        fq.fp8_gated_block_backward(dh, gu, sgu, h_t=_u8(130, 6), scale_inv_h_t=torch.zeros(130, 1))


@pytest.mark.parametrize("act", [G.SILU, G.GELU])
def test_reference_slope_against_differences(act):
    g = torch.cat([torch.linspace(-40, 40, 4001, dtype=torch.float64), torch.tensor([0.0, -0.0, 1e-30, -1e-30])])
    e = 1e-5
    a, slope, _, _ = G.activation(g, act)
    differences = (G.activation(g + e, act)[0] - G.activation(g - e, act)[0]) / (2 * e)
    # e^2 / 6 times a third derivative below 3, and 2^-52 |g| / e of rounding
    assert ((slope - differences).abs() < 5e-11 + 2.0 ** -52 * (g.abs() + 1) / e).all()
    # the definitions as they are usually written
    usual = g / (1 + torch.exp(-g)) if act == G.SILU else 0.5 * g * (1 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g ** 3)))
    assert ((a - usual).abs() <= 1e-13 * (1 + g.abs())).all()
    assert slope.abs().max() < 1.2


def test_gated_block_step_refuses_and_accounts():
    from fp8_scaled_quantization_gb300 import pipelines as P
    meta = torch.device("meta")
    mk = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=meta)  # noqa: E731
    ends = torch.empty(2, dtype=torch.int64, device=meta)
    with pytest.raises(ValueError, match="group_ends"):
        P.GatedBlockStep(mk(8, 256), mk(2, 2, 128, 256), mk(2, 256, 128), mk(8, 256))
    with pytest.raises(ValueError, match="group_ends"):
        P.GatedBlockStep(mk(8, 256), mk(2, 128, 256), mk(256, 128), mk(8, 256), ends)
    with pytest.raises(ValueError, match="gate_up must be"):
        P.GatedBlockStep(mk(8, 256), mk(3, 128, 256), mk(256, 128), mk(8, 256))
    with pytest.raises(ValueError, match="gate_up must be"):
        P.GatedBlockStep(mk(8, 256), mk(2, 128, 256), mk(128, 256), mk(8, 256))
    with pytest.raises(ValueError, match="multiple of 128"):
        P.GatedBlockStep(mk(8, 256), mk(2, 100, 256), mk(256, 100), mk(8, 256))
    with pytest.raises(ValueError, match="multiple of 128"):
        P.GatedBlockStep(mk(8, 200), mk(2, 2, 128, 200), mk(2, 200, 128), mk(8, 200), ends)
    b = P.GatedBlockStep(mk(512, 256), mk(2, 128, 256), mk(256, 128), mk(512, 256)).bytes()
    t, k, n = 512, 256, 128
    assert b.per_kernel["forward"] == (t * k + 4 * t * 2 + 2 * n * k + 4 * 4 + 3 * (t * n + 4 * t), 1)
    assert b.per_kernel["backward"] == (t * n * (2 + 2 + 2 + 2 + 1) + 4 * t * 4 + 4 * 3 * n * 4, 1)
    assert b.per_kernel["dx"] == (2 * t * n + 4 * 2 * t + 2 * n * k + 4 * 4 + 2 * t * k, 1)
    assert b.per_kernel["clip"] == (3 * n * k * 8, 1) and b.launches == 12
