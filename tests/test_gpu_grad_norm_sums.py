"""How well the gradient norm's sums hold over long tensors, aligned or not.

Per CTA the kernel takes `reps` chunks of 32 KB, reps = all chunks / (16 x SMs) above 16 x
SMs chunks.  A thread adds squares in four fp32 sums of at most 16 values, joins the four
(two additions) and adds the results of its chunks one after another: (16 + 2 + reps)
roundings of 2^-24 at most, sums of positive numbers, then 64 bits.  The square root halves
the relative error and the norm is rounded once: ((18 + reps) / 2 + 1) * 2^-24.
"""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def chunks(n, size):
    return -(-n * size // 32768)


def bound(total_chunks):
    many = 16 * torch.cuda.get_device_properties(0).multi_processor_count
    reps = total_chunks // many if total_chunks > many else 1
    return ((18 + reps) / 2 + 1) * 2.0 ** -24


def norm_of(xs):
    out = torch.empty(1, device=DEV)
    fq.fp8_grad_norm_grouped(xs, out)
    return out.item()


@pytest.mark.parametrize("shift", [0, 1])
def test_equal_values(shift):
    """3 GB of one value whose square is rounded to the same side in nearly every addition
    of a long fp32 sum; aligned, and one element off."""
    n, value = 37 * 16 * 152 * 8192 + 5, 1.8422846
    flat = torch.full((n + 1,), value, device=DEV)
    value = flat[0].item()
    norm, want = norm_of([flat[shift:shift + n]]), value * n ** 0.5
    assert abs(norm - want) <= bound(chunks(n, 4)) * want


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("dtype,n", [
    (torch.bfloat16, 6000 * 16384 + 77),   # two or three chunks per CTA
    (torch.float32, 5000 * 8192 - 1),
    (torch.bfloat16, 8000 * 16384),
    (torch.bfloat16, 300_000_001),
])
def test_random_values(dtype, n, shift):
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    x = torch.randn(n + 8, generator=g, device=DEV).to(dtype)[shift:shift + n]
    want = float((x.double() ** 2).sum().sqrt())
    assert abs(norm_of([x]) - want) <= bound(chunks(n, x.element_size())) * want
    y = torch.empty(n + 8, dtype=dtype, device=DEV)[shift:shift + n]
    norm, coef = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    fq.fp8_grad_clip_grouped([x], want / 3, norm, ys=[y], coef_out=coef)
    assert norm.item() == norm_of([x])
    assert torch.equal(y, (x.float() * coef).to(dtype))
