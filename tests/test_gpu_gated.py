"""The gated feed-forward block on the GPU against the plain 64-bit reference."""
from __future__ import annotations

import math

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gated_reference as G
import gemm_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CANARY = 0xA5


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


class Out:
    """Codes or factors between canaries, `shift` elements off a 64-byte boundary."""

    def __init__(self, shape, dtype=torch.uint8, shift=0):
        size = math.prod(shape)
        self.flat = torch.full((size + 128 + shift,), CANARY if dtype == torch.uint8 else -7.0, dtype=dtype, device=DEV)
        self.at, self.size = 64 + shift, size
        self.t = self.flat[self.at:self.at + size].view(shape)

    def intact(self):
        edges = torch.cat([self.flat[:self.at], self.flat[self.at + self.size:]])
        return bool((edges == self.flat[0]).all()) and self.flat[0].item() in (CANARY, -7.0)


def outputs(m, n, keep, shift=0):
    nb = G.blocks(n)
    outs = [Out((m, n), shift=shift), Out((m, nb), torch.float32)]
    if keep:
        outs += [Out((m, 2, n), shift=shift), Out((m, 2, nb), torch.float32)]
    return outs


def operands(m, n, k, seed, experts=None, fmt_a=R.E4M3, size=2.0):
    """Codes over the whole range; projections of about `size`."""
    g, kb, nb = gen(seed), G.blocks(k), G.blocks(n)
    lead = () if experts is None else (experts,)
    a = R.finite_codes((m, k), fmt_a, g, DEV)
    b = R.finite_codes((*lead, 2, n, k), R.E4M3, g, DEV)
    rms = [R.decode_table(f)[torch.arange(0x7F if f == R.E4M3 else 0x7C)].square().mean().sqrt().item() for f in (fmt_a, R.E4M3)]
    sa = torch.exp(torch.randn((m, kb), generator=g, device=DEV) * 0.5) / rms[0]
    sb = torch.exp(torch.randn((*lead, 2, nb, kb), generator=g, device=DEV) * 0.3) / rms[1] * size / math.sqrt(max(k, 1))
    return a, sa, b, sb


def projections(a, sa, b, sb, fmt_a=R.E4M3, fmt_b=R.E4M3):
    """[m, 2, n] of both and their bounds."""
    av = R.values(a, sa, fmt_a, 1)
    both = [R.product(av, R.values(b[i], sb[i], fmt_b, 128)) for i in (0, 1)]
    return torch.stack([v for v, _ in both], 1), torch.stack([e for _, e in both], 1)


def check(outs, gu, bound, act):
    h, eh = G.gated(gu[:, 0], gu[:, 1], bound[:, 0], bound[:, 1], act)
    G.check_tiles(outs[0].t, outs[1].t, h, eh, R.E4M3)
    if len(outs) > 2:
        G.check_tiles(outs[2].t, outs[3].t, gu, bound, R.E4M3)
    assert all(o.intact() for o in outs), "bytes beside an output"


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 16, 16), (3, 130, 129), (1, 7, 640), (5, 300, 144), (16, 128, 256), (17, 257, 384),
          (33, 129, 5000), (64, 256, 1024), (65, 272, 1040), (100, 384, 48), (128, 128, 128), (129, 512, 2048),
          (200, 1000, 1000), (255, 256, 512), (257, 513, 272), (300, 640, 1500), (512, 768, 1536), (1, 2048, 16),
          (1024, 16, 128), (1030, 1040, 656), (48, 4096, 1152), (7, 1536, 5120), (24, 144, 2048), (90, 4100, 700)]


@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gated(m, n, k, act):
    for keep, fmt_a in ((True, R.E4M3), (False, R.E5M2)):
        ops = operands(m, n, k, m + 3 * n + 7 * k, fmt_a=fmt_a)
        outs = outputs(m, n, keep)
        fq.fp8_gemm_block_gated(*ops, *[o.t for o in outs], fmt_a=fmt_a, act=act)
        check(outs, *projections(*ops, fmt_a=fmt_a), act)


@pytest.mark.parametrize("size", [1e-6, 30.0, 1e4])
@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("m", [9, 40, 300])
def test_small_and_saturated_projections(m, act, size):
    ops = operands(m, 384, 512, 3, size=size)
    outs = outputs(m, 384, True)
    fq.fp8_gemm_block_gated(*ops, *[o.t for o in outs], act=act)
    check(outs, *projections(*ops), act)


@pytest.mark.parametrize("m", [3, 40, 100, 280])
@pytest.mark.parametrize("shift", [1, 4])
def test_outputs_and_operands_that_start_anywhere(m, shift):
    n, k = 272, 400
    a, sa, b, sb = operands(m, n, k, 5)
    moved = [Out(t.shape, shift=shift) for t in (a, b)]
    for o, t in zip(moved, (a, b)):
        o.t.copy_(t)
    outs = outputs(m, n, True, shift)
    fq.fp8_gemm_block_gated(moved[0].t, sa, moved[1].t, sb, *[o.t for o in outs])
    check(outs, *projections(a, sa, b, sb), G.SILU)


@pytest.mark.parametrize("m", [2, 50, 300])
def test_no_contraction_gives_zeros(m):
    outs = outputs(m, 200, True)
    empty = [torch.empty(s, dtype=d, device=DEV) for s, d in (((m, 0), torch.uint8), ((m, 0), torch.float32),
                                                              ((2, 200, 0), torch.uint8), ((2, 2, 0), torch.float32))]
    fq.fp8_gemm_block_gated(*empty, *[o.t for o in outs])
    assert all(not (o.t & 0x7F).any() for o in outs[::2]) and all((o.t == 1).all() for o in outs[1::2])
    assert all(o.intact() for o in outs)


@pytest.mark.parametrize("m", [4, 30, 60, 290])
@pytest.mark.parametrize("act", [G.SILU, G.GELU])
def test_nan_and_infinity(m, act):
    """NaN codes and factors, and E5M2 infinities, reach the tiles that they belong to and no other."""
    n, k = 400, 384
    a, sa, b, sb = operands(m, n, k, 11, fmt_a=R.E5M2)
    a[1, 7] = 0x7F           # a row of NaN
    a[2, 300] = 0x7C         # a row of Inf, NaN where the weight is 0
    a[m - 1, 5] = 0xFC
    b[0, 130, 9] = 0x7F      # a column of the gate
    b[1, n - 1, 200] = 0xFF  # and of the up projection
    b[:, 260, 300] = 0
    outs = outputs(m, n, True)
    fq.fp8_gemm_block_gated(a, sa, b, sb, *[o.t for o in outs], fmt_a=R.E5M2, act=act)
    check(outs, *projections(a, sa, b, sb, fmt_a=R.E5M2), act)
    sb[0, 2, 1] = float("nan")
    fq.fp8_gemm_block_gated(a, sa, b, sb, *[o.t for o in outs], fmt_a=R.E5M2, act=act)
    check(outs, *projections(a, sa, b, sb, fmt_a=R.E5M2), act)


def grouped_check(ops, counts, outs, act):
    a, sa, b, sb = ops
    n, start = b.shape[-2], 0
    gu = torch.zeros((a.shape[0], 2, n), dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(gu)
    for e, c in enumerate(counts):
        if c:
            r = slice(start, start + c)
            gu[r], bound[r] = projections(a[r], sa[r], b[e], sb[e])
        start += c
    # (rows of no expert: zeros, with a bound of zero)
    check_rows = [Slice(o, start) for o in outs]
    h, eh = G.gated(gu[:, 0], gu[:, 1], bound[:, 0], bound[:, 1], act)
    G.check_tiles(outs[0].t[:start], outs[1].t[:start], h[:start], eh[:start], R.E4M3)
    if len(outs) > 2:
        G.check_tiles(outs[2].t[:start], outs[3].t[:start], gu[:start], bound[:start], R.E4M3)
    assert all(s.untouched_by_experts() for s in check_rows) and all(o.intact() for o in outs)


class Slice:
    def __init__(self, out, start):
        self.rest = out.t[start:]

    def untouched_by_experts(self):
        r = self.rest
        return bool(((r & 0x7F) == 0).all() if r.dtype == torch.uint8 else (r == 1).all())


COUNTS = [([5], 0), ([1, 0, 3], 2), ([0, 0, 0], 7), ([16, 17, 1, 0, 30], 0), ([300, 0, 129, 1, 255], 13), ([64] * 8, 0),
          ([0, 700], 0), ([2] * 40, 5), ([128, 128], 128)]


@pytest.mark.parametrize("counts,spare", COUNTS)
@pytest.mark.parametrize("n,k", [(256, 384), (200, 1040), (1, 100), (640, 2048)])
def test_experts(counts, spare, n, k):
    rows = sum(counts) + spare
    ops = operands(rows, n, k, rows + n + k, len(counts))
    ends = torch.tensor(counts, dtype=torch.int64, device=DEV).cumsum(0)
    for keep, act in ((True, G.SILU), (False, G.GELU)):
        outs = outputs(rows, n, keep)
        fq.fp8_gemm_block_gated_grouped(*ops, ends, *[o.t for o in outs], act=act)
        grouped_check(ops, counts, outs, act)


def test_ends_that_are_no_ends():
    """Out of range or falling group ends are taken as the nearest allowed value."""
    rows, n, k = 90, 256, 256
    ops = operands(rows, n, k, 1, 4)
    outs = outputs(rows, n, True)
    fq.fp8_gemm_block_gated_grouped(*ops, torch.tensor([-5, 40, 30, 10 ** 12], device=DEV), *[o.t for o in outs])
    grouped_check(ops, [0, 40, 0, 50], outs, G.SILU)


@pytest.mark.parametrize("m,n,k", [(1, 1, 2300), (7, 160, 2300), (33, 300, 2300), (64, 129, 2300), (16, 2048, 1024),
                                   (300, 520, 700), (128, 400, 2300)])
def test_calls_one_after_another_give_the_same(m, n, k):
    """Also the ends of the kernels, where CTAs of a cluster leave."""
    ops = operands(m, n, k, m + n)
    runs = [outputs(m, n, True) for _ in range(30)]
    for outs in runs:
        fq.fp8_gemm_block_gated(*ops, *[o.t for o in outs])
    check(runs[0], *projections(*ops), G.SILU)
    assert all(torch.equal(a.flat, b.flat) for outs in runs[1:] for a, b in zip(outs, runs[0]))


# ---------------------------------------------------------------- backward

def checkpoint(rows, n, seed, size=1.0):
    g = gen(seed)
    gu = R.finite_codes((rows, 2, n), R.E4M3, g, DEV)
    sgu = torch.exp(torch.randn((rows, 2, G.blocks(n)), generator=g, device=DEV) * 0.5) / 100.0 * size
    return gu, sgu


def gradient_outputs(rows, n, shift=0):
    nb, rb = G.blocks(n), G.blocks(rows)
    return [Out((rows, 2, n), shift=shift), Out((rows, 2, nb), torch.float32), Out((2, n, rows), shift=shift),
            Out((2, n, rb), torch.float32), Out((n, rows), shift=shift), Out((n, rb), torch.float32)]


def check_backward(outs, dh, gu, sgu, act, fmt):
    g, u = (R.values(gu[:, i], sgu[:, i], R.E4M3, 1) for i in (0, 1))
    (dg, eg), (du, eu), (h, eh) = G.backward(dh.double(), g, u, act)
    if outs[0] is not None:
        for i, (v, e) in enumerate(((dg, eg), (du, eu))):
            G.check_tiles(outs[0].t[:, i], outs[1].t[:, i], v, e, fmt)
    if outs[2] is not None:
        for i, (v, e) in enumerate(((dg, eg), (du, eu))):
            G.check_tiles(outs[2].t[i], outs[3].t[i], v.T, e.T, fmt)
    if outs[4] is not None:
        G.check_tiles(outs[4].t, outs[5].t, h.T, eh.T, R.E4M3)
    assert all(o.intact() for o in outs if o is not None), "bytes beside an output"


def back(dh, gu, sgu, outs, **kw):
    fq.fp8_gated_block_backward(dh, gu, sgu, *[o.t if o is not None else None for o in outs], **kw)


BACK_SHAPES = [(1, 1), (1, 128), (128, 1), (3, 130), (17, 1024), (128, 128), (129, 256), (127, 255), (256, 400), (300, 4),
               (260, 516), (16, 16), (144, 2064), (1000, 640), (513, 1001), (130, 2046), (2049, 384), (128, 8192)]


@pytest.mark.parametrize("act", [G.SILU, G.GELU])
@pytest.mark.parametrize("rows,n", BACK_SHAPES)
def test_backward(rows, n, act):
    for dtype, fmt in ((torch.bfloat16, R.E4M3), (torch.float32, R.E5M2), (torch.bfloat16, R.E5M2), (torch.float32, R.E4M3)):
        dh = (torch.randn((rows, n), generator=gen(rows * n), device=DEV) * 1e-2).to(dtype)
        gu, sgu = checkpoint(rows, n, rows + n)
        outs = gradient_outputs(rows, n)
        back(dh, gu, sgu, outs, fmt_grad=fmt, act=act)
        check_backward(outs, dh, gu, sgu, act, fmt)


@pytest.mark.parametrize("which", [(0, 1), (2, 3), (4, 5), (0, 1, 4, 5), (2, 3, 4, 5)])
@pytest.mark.parametrize("rows,n", [(256, 256), (77, 130), (1500, 384)])
def test_backward_outputs_that_are_left_out(rows, n, which):
    dh = torch.randn((rows, n), generator=gen(1), device=DEV).bfloat16()
    gu, sgu = checkpoint(rows, n, 2)
    outs = [o if i in which else None for i, o in enumerate(gradient_outputs(rows, n))]
    back(dh, gu, sgu, outs)
    check_backward(outs, dh, gu, sgu, G.SILU, R.E4M3)


@pytest.mark.parametrize("shift", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("rows,n", [(256, 256), (200, 144)])
def test_backward_arrays_that_start_anywhere(rows, n, shift):
    gu, sgu = checkpoint(rows, n, 2)
    moved = Out(gu.shape, shift=shift)
    moved.t.copy_(gu)
    for dtype in (torch.bfloat16, torch.float32):
        dh = Out((rows, n), dtype, shift)
        dh.t.copy_(torch.randn((rows, n), generator=gen(1), device=DEV))
        outs = gradient_outputs(rows, n, shift)
        back(dh.t, moved.t, sgu, outs)
        check_backward(outs, dh.t, gu, sgu, G.SILU, R.E4M3)


@pytest.mark.parametrize("size", [1e-30, 1e-4, 30.0, 1e6])
@pytest.mark.parametrize("act", [G.SILU, G.GELU])
def test_backward_of_small_and_saturated_projections(act, size):
    dh = torch.randn((200, 384), generator=gen(1), device=DEV)
    gu, sgu = checkpoint(200, 384, 2, size)
    outs = gradient_outputs(200, 384)
    back(dh, gu, sgu, outs, act=act, fmt_grad=R.E5M2)
    check_backward(outs, dh, gu, sgu, act, R.E5M2)


@pytest.mark.parametrize("fmt", [R.E4M3, R.E5M2])
@pytest.mark.parametrize("rows,n", [(256, 256), (133, 300)])
def test_backward_nan_infinity_and_zeros(rows, n, fmt):
    dh = torch.randn((rows, n), generator=gen(1), device=DEV).bfloat16()
    gu, sgu = checkpoint(rows, n, 2)
    dh[3, 5], dh[130, 200], dh[40, n - 1] = float("inf"), float("nan"), float("-inf")
    gu[7, 0, 9], gu[rows - 1, 1, 140] = 0x7F, 0xFF
    dh[20], gu[21] = 0, 0      # rows of zeros
    dh[:, 30], gu[:, :, 31] = 0, 0x80  # and columns
    sgu[50, 0, 1] = float("inf")
    outs = gradient_outputs(rows, n)
    back(dh, gu, sgu, outs, fmt_grad=fmt)
    check_backward(outs, dh, gu, sgu, G.SILU, fmt)


def test_past_32_bits():
    """Elements beyond 2^32 of the checkpoint and of the transposed gradients."""
    rows, n = 120016, 18432
    gu = torch.zeros((rows, 2, n), dtype=torch.uint8, device=DEV)
    sgu, dh = torch.ones((rows, 2, n // 128), device=DEV), torch.zeros((rows, n), dtype=torch.bfloat16, device=DEV)
    r = slice(rows - 200, rows)
    part, spart = checkpoint(200, n, 4)
    gu[r], sgu[r] = part, spart
    dh[r] = torch.randn((200, n), generator=gen(1), device=DEV).bfloat16()
    rb = G.blocks(rows)
    dgu, sdgu, dgu_t, sdgu_t = (torch.full(s, 9, dtype=d, device=DEV) for s, d in (
        ((rows, 2, n), torch.uint8), ((rows, 2, n // 128), torch.float32), ((2, n, rows), torch.uint8),
        ((2, n, rb), torch.float32)))
    fq.fp8_gated_block_backward(dh, gu, sgu, dgu, sdgu, dgu_t, sdgu_t)
    g, u = (R.values(gu[r, i], sgu[r, i], R.E4M3, 1) for i in (0, 1))
    (dg, eg), (du, eu), _ = G.backward(dh[r].double(), g, u, G.SILU)
    first = (rows - 200 + 127) // 128 * 128 - (rows - 200)  # from the first tile that lies in these rows whole
    for i, (v, e) in enumerate(((dg, eg), (du, eu))):
        G.check_tiles(dgu[r, i], sdgu[r, i], v, e, R.E4M3)
        G.check_tiles(dgu_t[i][:, rows - 200 + first:], sdgu_t[i][:, (rows - 200 + first) // 128:], v[first:].T, e[first:].T, R.E4M3)
    assert (sdgu[:rows - 200] == 1).all() and not (dgu[:64] & 0x7F).any()


def test_more_rows_than_half_of_32_bits():
    """Rows of both projections beyond 2^31: one column, of which the last rows are looked at."""
    rows = 2 ** 30 + 300
    gu, sgu = torch.zeros((rows, 2, 1), dtype=torch.uint8, device=DEV), torch.ones((rows, 2, 1), device=DEV)
    dh = torch.zeros((rows, 1), dtype=torch.bfloat16, device=DEV)
    r = slice(rows - 300, rows)
    gu[r], sgu[r] = checkpoint(300, 1, 4)
    dh[r] = torch.randn((300, 1), generator=gen(1), device=DEV).bfloat16()
    dgu, sdgu = torch.full((rows, 2, 1), 9, dtype=torch.uint8, device=DEV), torch.zeros((rows, 2, 1), device=DEV)
    dgu_t, sdgu_t = torch.full((2, 1, rows), 9, dtype=torch.uint8, device=DEV), torch.zeros((2, 1, G.blocks(rows)), device=DEV)
    fq.fp8_gated_block_backward(dh, gu, sgu, dgu, sdgu, dgu_t, sdgu_t)
    g, u = (R.values(gu[r, i], sgu[r, i], R.E4M3, 1) for i in (0, 1))
    (dg, eg), (du, eu), _ = G.backward(dh[r].double(), g, u, G.SILU)
    first = -(rows - 300) % 128  # from the first tile of a column that lies in these rows whole
    for i, (v, e) in enumerate(((dg, eg), (du, eu))):
        G.check_tiles(dgu[r, i], sdgu[r, i], v, e, R.E4M3)
        G.check_tiles(dgu_t[i][:, rows - 300 + first:], sdgu_t[i][:, (rows - 300 + first) // 128:], v[first:].T, e[first:].T, R.E4M3)
    assert (sdgu[:2 ** 20] == 1).all() and not (dgu_t[:, :, :2 ** 20] & 0x7F).any()


# ---------------------------------------------------------- streams and graphs

def test_on_a_stream_and_in_a_graph():
    m, n, k = 140, 384, 512
    ops = operands(m, n, k, 9)
    dh = torch.randn((m, n), generator=gen(1), device=DEV).bfloat16()
    outs, grads = outputs(m, n, True), gradient_outputs(m, n)

    def both():
        fq.fp8_gemm_block_gated(*ops, *[o.t for o in outs])
        back(dh, outs[2].t, outs[3].t, grads)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    first = [o.flat.clone() for o in outs + grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for o in outs + grads:
        o.t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, o.flat) for a, o in zip(first, outs + grads))
    check(outs, *projections(*ops), G.SILU)
    check_backward(grads, dh, outs[2].t, outs[3].t, G.SILU, R.E4M3)


def test_threads_and_streams_at_once():
    """Calls that copy odd operands into their stream's scratch, from four host threads on three
    streams (two threads share one), give what they give alone."""
    import threading
    shapes = [(3, 300, 515), (70, 257, 770), (260, 520, 333), (40, 130, 901)]
    ops = [operands(*s, i + 1) for i, s in enumerate(shapes)]
    alone, failed = [], []

    def call(i, outs, grads):
        fq.fp8_gemm_block_gated(*ops[i], *[o.t for o in outs])
        back(outs[0].t.bfloat16(), outs[2].t, outs[3].t, grads)

    fresh = lambda i: (outputs(*shapes[i][:2], True), gradient_outputs(*shapes[i][:2]))  # noqa: E731
    for i in range(4):
        alone.append(fresh(i))
        call(i, *alone[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]

    def work(i):
        try:
            with torch.cuda.stream(streams[i % 3]):
                for _ in range(20):
                    outs, grads = fresh(i)
                    call(i, outs, grads)
                    streams[i % 3].synchronize()
                    if not all(torch.equal(a.flat, b.flat) for a, b in zip(outs + grads, alone[i][0] + alone[i][1])):
                        failed.append(i)
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed


def test_a_captured_call_keeps_its_scratch():
    """Odd operands of a captured call: larger eager calls on the stream leave the graph's copy alone."""
    small, large = operands(20, 200, 331, 1), operands(300, 1000, 1501, 2)
    a, b = outputs(20, 200, False), outputs(300, 1000, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fq.fp8_gemm_block_gated(*small, *[o.t for o in a])
    s.synchronize()
    first = [o.flat.clone() for o in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fq.fp8_gemm_block_gated(*small, *[o.t for o in a])
    with torch.cuda.stream(s):
        fq.fp8_gemm_block_gated(*large, *[o.t for o in b])
    for o in a:
        o.t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, o.flat) for x, o in zip(first, a))
    check(b, *projections(*large), G.SILU)
