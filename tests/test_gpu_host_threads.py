"""Several host threads on one stream: calls that write the stream's workspace or scratch
in one launch and read it in the next must not mix.  Every thread's results are the bits
of the same calls made alone."""
from __future__ import annotations

import threading

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gemm_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CALLS = 300


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def race(jobs):
    """jobs: per thread a function of the call's number that returns nothing; all on the current stream."""
    start, errors = threading.Barrier(len(jobs)), []

    def work(job):
        try:
            torch.cuda.set_device(0)
            start.wait(30)
            for i in range(CALLS):
                job(i)
        except Exception as e:  # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()


@pytest.mark.parametrize("m,n,k", [(5, 256, 333), (600, 520, 333)])
def test_products_with_odd_rows(m, n, k):
    """Both kernels; the two threads' operands have the same sizes, so that they share the scratch's bytes."""
    jobs, outs, wants = [], [], []
    for seed in (1, 2, 3):
        g = gen(seed)
        kb, nb = -(-k // 128), -(-n // 128)
        a, sa = R.finite_codes((m, k), 0, g, DEV), R.scales((m, kb), g, DEV)
        b, sb = R.finite_codes((n, k), 0, g, DEV), R.scales((nb, kb), g, DEV)
        alone, d = torch.empty((m, n), device=DEV), torch.empty((CALLS, m, n), device=DEV)
        fq.fp8_gemm_block(a, sa, b, sb, alone)
        jobs.append(lambda i, a=a, sa=sa, b=b, sb=sb, d=d: fq.fp8_gemm_block(a, sa, b, sb, d[i]))
        outs.append(d)
        wants.append(alone)
    race(jobs)
    for d, w in zip(outs, wants):
        assert (d == w).all()


def test_norms_clips_and_amaxes():
    """Every kind of call that reduces through the workspace, at once."""
    jobs, checks = [], []

    def norm(seed, sizes):
        xs = [torch.randn(n, generator=gen(seed), device=DEV) for n in sizes]
        out, alone = torch.empty((CALLS, 1), device=DEV), torch.empty(1, device=DEV)
        fq.fp8_grad_norm_grouped(xs, alone)
        jobs.append(lambda i: fq.fp8_grad_norm_grouped(xs, out[i]))
        checks.append((out, alone))

    def clip(seed, sizes):
        xs = [torch.randn(n, generator=gen(seed), device=DEV).bfloat16() for n in sizes]
        ys = [torch.empty_like(x) for x in xs]
        out, alone = torch.empty((CALLS, 2), device=DEV), torch.empty(2, device=DEV)
        fq.fp8_grad_clip_grouped(xs, 1.0, alone[:1], ys=ys, coef_out=alone[1:])
        jobs.append(lambda i: fq.fp8_grad_clip_grouped(xs, 1.0, out[i, :1], ys=ys, coef_out=out[i, 1:]))
        checks.append((out, alone))

    def amax(seed, n):
        x = torch.randn(n, generator=gen(seed), device=DEV) * seed
        out, alone = torch.empty((CALLS, 1), device=DEV), torch.empty(1, device=DEV)
        fq.fp8_amax(x, alone)
        jobs.append(lambda i: fq.fp8_amax(x, out[i]))
        checks.append((out, alone))

    def current(seed, n, odd):
        flat = torch.randn(n + 1, generator=gen(seed), device=DEV).bfloat16() * seed
        x = flat[odd:odd + n]
        q, one = torch.empty((CALLS, n), dtype=torch.uint8, device=DEV), torch.empty(n, dtype=torch.uint8, device=DEV)
        fq.fp8_quantize_current(x, fq.E4M3, one)
        jobs.append(lambda i: fq.fp8_quantize_current(x, fq.E4M3, q[i]))
        checks.append((q, one))

    norm(1, [100000, 77])
    clip(2, [4096, 3, 70001])
    clip(3, [30_000_000])
    amax(5, 1_000_000)
    current(7, 80_000, 0)
    current(9, 80_000, 1)
    race(jobs)
    for out, alone in checks:
        assert (out == alone).all()
