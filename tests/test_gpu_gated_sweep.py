"""Random sizes, groups, alignments, ranges and outputs of the gated feed-forward block and
its backward pass, against the plain 64-bit reference."""
from __future__ import annotations

import math
import random

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gated_reference as G
import gemm_reference as R
import test_gpu_gated as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def size(rng, lo, hi):
    """A size over the logarithm of [lo, hi]: a multiple of 128, 16 or 4, or any number."""
    v, kind = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), rng.random()
    step = 128 if kind < 0.3 else 16 if kind < 0.55 else 4 if kind < 0.7 else 1
    return max(lo, v // step * step or v)


@pytest.mark.parametrize("seed", range(40))
def test_gated(seed):
    rng = random.Random(seed)
    m, n, k = size(rng, 1, 900), size(rng, 1, 1500), size(rng, 1, 3000)
    act = rng.choice([G.SILU, G.GELU])
    ops = T.operands(m, n, k, seed, size=rng.choice([0.1, 2.0, 20.0]))
    outs = T.outputs(m, n, rng.random() < 0.5, rng.choice([0, 0, 1, 4]))
    fq.fp8_gemm_block_gated(*ops, *[o.t for o in outs], act=act)
    T.check(outs, *T.projections(*ops), act)


@pytest.mark.parametrize("seed", range(25))
def test_experts(seed):
    rng = random.Random(seed)
    counts = [rng.choice([0, 1, rng.randrange(1, 300), rng.randrange(1, 40)]) for _ in range(size(rng, 1, 40))]
    counts[-1] += 1
    rows, n, k = sum(counts) + rng.choice([0, 0, rng.randrange(1, 100)]), size(rng, 1, 600), size(rng, 1, 1500)
    act = rng.choice([G.SILU, G.GELU])
    ops = T.operands(rows, n, k, seed, len(counts))
    outs = T.outputs(rows, n, rng.random() < 0.5)
    fq.fp8_gemm_block_gated_grouped(*ops, torch.tensor(counts, device=T.DEV).cumsum(0), *[o.t for o in outs], act=act)
    T.grouped_check(ops, counts, outs, act)


@pytest.mark.parametrize("seed", range(50))
def test_backward(seed):
    rng = random.Random(seed)
    rows, n, shift = size(rng, 1, 2000), size(rng, 1, 2500), rng.choice([0, 0, 0, 1, 2, 4, 8])
    act, fmt, dtype = rng.choice([G.SILU, G.GELU]), rng.choice([R.E4M3, R.E5M2]), rng.choice([torch.bfloat16, torch.float32])
    gu, sgu = T.checkpoint(rows, n, seed, rng.choice([1e-3, 1.0, 10.0]))
    moved, dh = T.Out(gu.shape, shift=shift), T.Out((rows, n), dtype, shift)
    moved.t.copy_(gu)
    dh.t.copy_(torch.randn((rows, n), generator=T.gen(seed), device=T.DEV) * 10 ** rng.uniform(-6, 2))
    left_out = rng.choice([(), (), (0, 1), (2, 3), (4, 5), (0, 1, 2, 3)])
    outs = [None if i in left_out else o for i, o in enumerate(T.gradient_outputs(rows, n, shift))]
    T.back(dh.t, moved.t, sgu, outs, fmt_grad=fmt, act=act)
    T.check_backward(outs, dh.t, gu, sgu, act, fmt)
