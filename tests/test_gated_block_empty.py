"""A gated block's step without rows: what a rank whose experts got no token runs."""
from __future__ import annotations

import pytest
import torch

from fp8_scaled_quantization_gb300 import pipelines as P

IN, HIDDEN = 384, 256


def make(device, experts):
    mk = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=device)  # noqa: E731
    lead = () if experts is None else (experts,)
    ends = None if experts is None else torch.zeros(experts, dtype=torch.int64, device=device)
    return mk(0, IN), mk(*lead, 2, HIDDEN, IN), mk(*lead, IN, HIDDEN), mk(0, IN), ends


@pytest.mark.parametrize("experts", [None, 3])
def test_buffers_and_bytes(experts):
    step = P.GatedBlockStep(*make(torch.device("meta"), experts))
    assert [tuple(t.shape) for t in step.qx] == [(0, IN), (0, 3), (IN, 0), (IN, 0)]
    assert [tuple(t.shape) for t in step.grads] == [(0, 2, HIDDEN), (0, 2, 2), (2, HIDDEN, 0), (2, HIDDEN, 0),
                                                    (HIDDEN, 0), (HIDDEN, 0)]
    b, codes = step.bytes().per_kernel, HIDDEN * IN * (experts or 1)
    assert b["wgrad_gate_up"] == (2 * codes * 4, 1) and b["wgrad_down"] == (codes * 4, 1) and b["backward"] == (0, 1)


@pytest.mark.parametrize("experts", [None, 3])
def test_every_call_is_made(experts, monkeypatch):
    """The step reaches its last call, and the backward products get operands of their shapes."""
    calls = []
    for name in [n for n in vars(P) if n.startswith("fp8_")]:
        monkeypatch.setattr(P, name, lambda *a, name=name, **kw: calls.append((name, a)))
    P.GatedBlockStep(*make(torch.device("meta"), experts)).run()
    grouped = "" if experts is None else "_grouped"
    assert [c[0] for c in calls] == [
        "fp8_quantize_block", "fp8_quantize_block", "fp8_quantize_block_cast_transpose", "fp8_gemm_block_gated" + grouped,
        "fp8_gemm_block" + grouped, "fp8_quantize_block_cast_transpose", "fp8_gemm_block" + grouped,
        "fp8_gated_block_backward", "fp8_gemm_block" + grouped, *["fp8_gemm_block" + (grouped and "_grouped_wgrad")] * 2,
        "fp8_grad_clip_grouped"]
    shapes = lambda a, n: [tuple(t.shape) for t in a[:n]]  # noqa: E731
    lead = () if experts is None else (experts,)
    assert shapes(calls[8][1], 4) == [(0, 2 * HIDDEN), (0, 4), (*lead, 2 * HIDDEN, IN), (*lead, 4, 3)]  # dx
    assert shapes(calls[9][1], 4) == [(2 * HIDDEN, 0), (2 * HIDDEN, 0), (IN, 0), (IN, 0)]                # dWg, dWu
    assert shapes(calls[10][1], 4) == [(IN, 0), (IN, 0), (HIDDEN, 0), (HIDDEN, 0)]                       # dWd


@pytest.mark.gpu
@pytest.mark.parametrize("experts", [None, 3])
def test_run(cuda, experts):
    step = P.GatedBlockStep(*make(cuda, experts))
    step.dgate_up.fill_(5.0)
    step.ddown.fill_(5.0)
    step.norm.fill_(5.0)
    step.run()
    torch.cuda.synchronize()
    assert (step.dgate_up == 0).all() and (step.ddown == 0).all() and step.norm.item() == 0.0
