"""A layer's step without rows: what a rank whose experts got no token runs."""
from __future__ import annotations

import pytest
import torch

from fp8_scaled_quantization_gb300 import pipelines as P


def make(device, experts):
    mk = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=device)  # noqa: E731
    if experts is None:
        return mk(0, 384), mk(256, 384), mk(0, 256), None
    return mk(0, 384), mk(experts, 256, 384), mk(0, 256), torch.zeros(experts, dtype=torch.int64, device=device)


@pytest.mark.parametrize("experts", [None, 3])
def test_buffers_and_bytes(experts):
    step = P.BlockLinearStep(*make(torch.device("meta"), experts))
    assert [tuple(t.shape) for t in step.qx] == [(0, 384), (0, 3), (384, 0), (384, 0)]
    assert [tuple(t.shape) for t in step.qdy] == [(0, 256), (0, 2), (256, 0), (256, 0)]
    assert step.y.shape == (0, 256) and step.dx.shape == (0, 384)
    codes = 256 * 384 * (experts or 1)
    assert step.bytes().per_kernel["wgrad"] == (codes * 4, 1) and step.bytes().per_kernel["quantize_x"] == (0, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("experts", [None, 3])
def test_run(cuda, experts):
    step = P.BlockLinearStep(*make(cuda, experts))
    step.dweight.fill_(5.0)
    step.run()
    torch.cuda.synchronize()
    assert (step.dweight == 0).all() and step.norm.item() == 0.0
