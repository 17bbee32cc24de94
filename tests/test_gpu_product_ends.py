"""The ends of the block-scaled product kernels, where CTAs of a cluster leave: tiles
whose last columns are not there, so that some warps have nothing to store after their
last arrival, launched one after another, each result against the plain 64-bit one."""
from __future__ import annotations

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gemm_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


@pytest.fixture(autouse=True)
def _no_wait_gives_up(_built):
    before = fq.wait_timeouts()
    yield
    assert fq.wait_timeouts() == before


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def blocks(n):
    return -(-n // 128)


@pytest.mark.parametrize("m,n", [(1, 1), (300, 1), (256, 128), (129, 130), (520, 257), (700, 520)])
@pytest.mark.parametrize("counts", [[128], [1, 0, 127, 300], [256, 129, 640]])
def test_pairs_leave_after_each_others_last_arrivals(m, n, counts):
    """Ragged contractions always take CTA pairs; n is at most 128 columns beyond a tile of 256."""
    rows, e, g = sum(counts), len(counts), gen(m + n)
    a, sa = R.finite_codes((m, rows), 1, g, DEV), R.scales((m, blocks(rows)), g, DEV)
    b, sb = R.finite_codes((n, rows), 0, g, DEV), R.scales((n, blocks(rows)), g, DEV)
    ends = torch.tensor(counts, dtype=torch.int64, device=DEV).cumsum(0)
    ds = [torch.full((e, m, n), float("nan"), device=DEV) for _ in range(40)]
    for d in ds:
        fq.fp8_gemm_block_grouped_wgrad(a, sa, b, sb, ends, d, fq.E5M2, fq.E4M3)
    av, bv, start = R.values(a, sa, 1, 1), R.values(b, sb, 0, 1), 0
    for i, c in enumerate(counts):
        value, bound = R.product(av[:, start:start + c], bv[:, start:start + c])
        # a group that is not aligned to 128 touches up to two blocks more than its length says
        R.check(ds[0][i], value, bound * (128 + blocks(c) + 6) / (128 + blocks(c) + 4))
        start += c
    assert all(torch.equal(d, ds[0]) for d in ds[1:])


@pytest.mark.parametrize("form", ["nk", "kn", "tiles"])
@pytest.mark.parametrize("m", [1, 7, 16, 33, 64, 100])
@pytest.mark.parametrize("n", [1, 32, 33, 129, 160, 300])
def test_clusters_leave_after_reads_of_each_others_sums(n, m, form):
    """Few columns and a long contraction: as many CTAs share it as a cluster holds, and in
    the last 128 columns whole warps have no column to join."""
    k, g = 2300, gen(n + m)
    a, sa = R.finite_codes((m, k), 0, g, DEV), R.scales((m, blocks(k)), g, DEV)
    shape, scales = {"nk": ((n, k), (blocks(n), blocks(k))), "kn": ((k, n), (blocks(k), blocks(n))),
                     "tiles": ((n, k), (n, blocks(k)))}[form]
    b, sb = R.finite_codes(shape, 0, g, DEV), R.scales(scales, g, DEV)
    ds = [torch.full((m, n), float("nan"), device=DEV) for _ in range(40)]
    for d in ds:
        fq.fp8_gemm_block(a, sa, b, sb, d, b_layout=fq.B_KN if form == "kn" else fq.B_NK,
                          b_block_rows=1 if form == "tiles" else 128)
    bv = R.values(b, sb, 0, 1 if form == "tiles" else 128)
    R.check(ds[0], *R.product(R.values(a, sa, 0, 1), bv.T if form == "kn" else bv))
    assert all(torch.equal(d, ds[0]) for d in ds[1:])


def test_a_group_end_behind_a_long_contraction():
    """8e8 rows of one expert, four seconds for one CTA pair: the block that its end cuts is
    masked only then, and what waits for that block must not have given up."""
    rows = 3 * 2 ** 28
    ends = [rows - 200, rows - 75, rows]
    a, b = (torch.zeros((1, rows), dtype=torch.uint8, device=DEV) for _ in range(2))
    one = 0x38  # 1.0 in E4M3: every sum below is exact
    at = torch.cat([torch.arange(0, rows - 300, 2 ** 20 + 7), torch.arange(rows - 290, rows)]).to(DEV)
    a[0, at], b[0, at] = one, one
    a[0, rows - 150], b[0, rows - 40] = 0x7F, 0x7F  # NaN in groups 1 and 2 only
    scale = torch.ones((1, blocks(rows)), device=DEV)
    d = torch.empty((3, 1, 1), device=DEV)
    fq.fp8_gemm_block_grouped_wgrad(a, scale, b, scale, torch.tensor(ends, device=DEV), d)
    torch.cuda.synchronize()
    assert d[0].item() == int((at < ends[0]).sum()) and d[1].isnan().all() and d[2].isnan().all()
