"""The gated block's kernels after their first tile: sizes at which each CTA, pair or cluster takes
several, so that loading ahead, alternating buffers and the last tile's stores beside the next are
reached in every form; all elements checked."""
from __future__ import annotations

import math
import random

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gated_bounds as B
import gated_reference as G
import gemm_reference as R
import test_gpu_gated as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


@pytest.fixture(autouse=True)
def _no_wait_gives_up(_built):
    before = fq.wait_timeouts()
    yield
    assert fq.wait_timeouts() == before


def run_back(rows, n, dtype, fmt, act, seed, shift=0, left_out=(), size=1.0):
    gu, sgu = T.checkpoint(rows, n, seed, size)
    moved, dh = T.Out(gu.shape, shift=shift), T.Out((rows, n), dtype, shift)
    moved.t.copy_(gu)
    dh.t.copy_(torch.randn((rows, n), generator=T.gen(seed + 1), device=T.DEV) * 1e-2)
    outs = [None if i in left_out else o for i, o in enumerate(T.gradient_outputs(rows, n, shift))]
    T.back(dh.t, moved.t, sgu, outs, fmt_grad=fmt, act=act)
    B.check_backward([o.t if o is not None else None for o in outs], dh.t, gu, sgu, act, fmt)
    assert all(o.intact() for o in outs if o is not None), "bytes beside an output"


# Tiles of 128 x 128, runs of four of them or of one by what fills 152 SMs better:
#  4096 x 7168: 32 x 56, runs of four, all aligned    4111 x 4230: 33 x 34, runs of four, the last of two
#  4100 x 4236: the same by words                      2560 x 2048: 20 x 16, single tiles, factors by four
#  2060 x 2564: 17 x 21, single tiles, by words        2563 x 2050: 21 x 17, unaligned single tiles
BACK = [(4096, 7168), (4111, 4230), (4100, 4236), (2560, 2048), (2060, 2564), (2563, 2050)]


@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("fmt", [R.E4M3, R.E5M2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", BACK)
def test_backward(rows, n, dtype, fmt, act):
    run_back(rows, n, dtype, fmt, act, rows + n)


@pytest.mark.parametrize("left_out", [(0, 1), (2, 3), (4, 5), (2, 3, 4, 5), (0, 1, 4, 5), (0, 1, 2, 3)])
@pytest.mark.parametrize("rows,n,dtype", [(4100, 4236, torch.bfloat16), (2560, 2048, torch.float32)])
def test_backward_outputs_that_are_left_out(rows, n, dtype, left_out):
    run_back(rows, n, dtype, R.E4M3, G.SILU, 5, left_out=left_out)


@pytest.mark.parametrize("seed", range(24))
def test_backward_random(seed):
    rng = random.Random(seed)

    def size():
        v, step = int(math.exp(rng.uniform(math.log(1500), math.log(5000)))), rng.choice([1, 1, 4, 16, 128])
        return v // step * step

    run_back(size(), size(), rng.choice([torch.bfloat16, torch.float32]), rng.choice([R.E4M3, R.E5M2]),
             rng.choice([G.SILU, G.GELU]), seed, rng.choice([0, 0, 0, 1, 2, 4, 8]),
             rng.choice([(), (), (0, 1), (2, 3), (4, 5)]), rng.choice([1e-3, 1.0, 30.0]))


# Rows, n, k: 256 x 128 tiles of the pair kernel beyond 76 pairs, then 16, 32 and 64 tokens by 128
# columns beyond 152 clusters of two.
FORWARD = [(2039, 2859, 400), (2000, 2864, 384), (1500, 4096, 1030), (20000, 144, 272), (1, 26852, 94), (3, 34848, 879),
           (23, 29233, 62), (20, 34224, 892), (35, 30400, 719), (36, 30761, 1702)]


@pytest.mark.parametrize("keep,act", [(True, G.SILU), (False, G.GELU), (True, G.GELU), (False, G.SILU)])
@pytest.mark.parametrize("m,n,k", FORWARD)
def test_forward(m, n, k, keep, act):
    ops = T.operands(m, n, k, m + n + k)
    outs = T.outputs(m, n, keep)
    fq.fp8_gemm_block_gated(*ops, *[o.t for o in outs], act=act)
    B.check_forward([o.t for o in outs], *T.projections(*ops), act)
    assert all(o.intact() for o in outs), "bytes beside an output"


@pytest.mark.parametrize("keep,act", [(True, G.GELU), (False, G.SILU)])
@pytest.mark.parametrize("counts,spare,n,k", [
    ([5, 0, 4, 1, 7, 2, 0, 3] * 2, 8, 1941, 61), ([11, 13, 0, 23], 3, 13663, 138), ([20, 17], 1, 18960, 20),
    ([300, 0, 257, 12, 1, 600, 255, 256], 40, 2320, 84), ([100] * 16, 0, 1300, 300)])
def test_experts(counts, spare, n, k, keep, act):
    rows = sum(counts) + spare
    ops = T.operands(rows, n, k, rows + n, len(counts))
    outs = T.outputs(rows, n, keep)
    fq.fp8_gemm_block_gated_grouped(*ops, torch.tensor(counts, device=T.DEV).cumsum(0), *[o.t for o in outs], act=act)
    T.grouped_check(ops, counts, outs, act)
