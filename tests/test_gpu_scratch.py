"""The scratch that products with odd rows copy their operands into: how much of it there
is after it has grown, and that captured graphs keep the part they were captured with."""
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


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def operands(m, n, k, seed):
    g, kb, nb = gen(seed), -(-k // 128), -(-n // 128)
    return (R.finite_codes((m, k), 0, g, DEV), R.scales((m, kb), g, DEV), R.finite_codes((n, k), 0, g, DEV),
            R.scales((nb, kb), g, DEV))


def want(a, sa, b, sb):
    return R.product(R.values(a, sa, 0, 1), R.values(b, sb, 0, 128))


def test_slow_growth_keeps_no_more_than_the_largest_call():
    """Weights of 8 MB to 1 GB in steps of 30%: outgrown buffers, 3.4 GB in all, do not stay."""
    m, n, ks = 4, 8192, [1001]
    while ks[-1] < 110000:
        ks.append(int(ks[-1] * 1.3) | 1)
    most = ks[-1]
    a, b = (torch.randint(0, 0x70, (r * most,), generator=gen(r), device=DEV, dtype=torch.uint8) for r in (m, n))
    s = R.scales((n // 128 * (most // 128 + 1),), gen(1), DEV)
    ds = torch.empty((len(ks), m, n), device=DEV)

    def call(i, k):
        kb = -(-k // 128)
        args = a[:m * k].view(m, k), s[:m * kb].view(m, kb), b[:n * k].view(n, k), s[:n // 128 * kb].view(-1, kb)
        fq.fp8_gemm_block(*args, ds[i])
        return args

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    with torch.cuda.stream(stream):
        args = [call(i, k) for i, k in enumerate(ks)]
    torch.cuda.synchronize()
    used = before - torch.cuda.mem_get_info()[0]
    largest = (m + n) * (most + 15)
    fq.release_stream_workspace(stream)
    assert used <= 1.25 * largest + 2 ** 27, f"{used / 2 ** 20:.0f} MiB held, largest call {largest / 2 ** 20:.0f}"
    for (qa, sa, qb, sb), d in zip(args, ds):
        r = slice(n - 256, n)
        value, bound = want(qa, sa, qb[r], sb[-2:])
        R.check(d[:, r], value, bound)


@pytest.mark.parametrize("first", [True, False])
def test_a_graph_keeps_its_scratch_when_later_calls_outgrow_it(first):
    """first: the stream has scratch before the capture; else the capture allocates it."""
    small, large = operands(20, 256, 333, 1), operands(300, 520, 1001, 2)
    d, big = torch.empty((20, 256), device=DEV), torch.empty((300, 520), device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if first:
        fq.fp8_gemm_block(*small, d, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fq.fp8_gemm_block(*small, d)
    for turn in range(3):
        d.zero_(), big.zero_()
        s.wait_stream(torch.cuda.current_stream())
        fq.fp8_gemm_block(*large, big, stream=s)
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        R.check(d, *want(*small))
        R.check(big, *want(*large))
        large = operands(300 + 300 * turn, 520, 1001 + 1000 * turn, 3)
        big = torch.empty((300 + 300 * turn, 520), device=DEV)
    del g
    fq.release_stream_workspace(s)


def test_growth_while_a_capture_is_under_way():
    """Two captured calls, the second larger: both addresses stay with the graph, and the
    buffer that the capture outgrew without using it is freed by the next plain call."""
    one, two, three = operands(20, 256, 333, 1), operands(40, 520, 1001, 2), operands(60, 520, 2001, 3)
    d1, d2, d3 = (torch.empty((o[0].shape[0], o[2].shape[0]), device=DEV) for o in (one, two, three))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fq.fp8_gemm_block(*operands(3, 16, 17, 4), torch.empty((3, 16), device=DEV), stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fq.fp8_gemm_block(*one, d1)
        fq.fp8_gemm_block(*two, d2)
    fq.fp8_gemm_block(*three, d3, stream=s)
    with torch.cuda.stream(s):
        g.replay()
    torch.cuda.synchronize()
    for o, d in ((one, d1), (two, d2), (three, d3)):
        R.check(d, *want(*o))
    del g
    fq.release_stream_workspace(s)
