"""Block-scaled FP8 products on the GPU against the plain 64-bit reference."""
from __future__ import annotations

import itertools

import pytest
import torch

import fp8_scaled_quantization_gb300 as fq
import gemm_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
OUTS = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built(native_lib):
    return native_lib


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def blocks(n):
    return -(-n // 128)


def operands(m, n, k, form, fmt_a, fmt_b, seed):
    """Codes and scales of one product; `form`: nk (weight), kn (weight read the other way), tiles (1 x 128 both)."""
    g = gen(seed)
    a, sa = R.finite_codes((m, k), fmt_a, g, DEV), R.scales((m, blocks(k)), g, DEV)
    if form == "kn":
        b, sb = R.finite_codes((k, n), fmt_b, g, DEV), R.scales((blocks(k), blocks(n)), g, DEV)
    else:
        b = R.finite_codes((n, k), fmt_b, g, DEV)
        sb = R.scales((n if form == "tiles" else blocks(n), blocks(k)), g, DEV)
    return a, sa, b, sb


def call(a, sa, b, sb, d, form, fmt_a, fmt_b, **kw):
    fq.fp8_gemm_block(a, sa, b, sb, d, fmt_a, fmt_b, b_layout=fq.B_KN if form == "kn" else fq.B_NK,
                      b_block_rows=1 if form == "tiles" else 128, **kw)


def want(a, sa, b, sb, form, fmt_a, fmt_b):
    av = R.values(a, sa, fmt_a, 1)
    bv = R.values(b, sb, fmt_b, 1 if form == "tiles" else 128)
    return R.product(av, bv.T if form == "kn" else bv)


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 16, 16), (3, 130, 129), (1, 7, 640), (5, 300, 144), (16, 128, 256),
          (17, 257, 384), (64, 256, 1024), (65, 272, 1040), (100, 384, 48), (128, 128, 128), (129, 512, 2048),
          (200, 1000, 1000), (255, 256, 512), (256, 256, 256), (257, 513, 272), (300, 640, 3000), (512, 768, 1536),
          (1, 2048, 16), (1024, 16, 128), (1030, 1040, 656), (48, 4096, 1152), (7, 1536, 5120), (33, 129, 9999)]


@pytest.mark.parametrize("form", ["nk", "kn", "tiles"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, form):
    for i, (fa, fb) in enumerate([(0, 0), (1, 0)]):
        ops = operands(m, n, k, form, fa, fb, m + 3 * n + 7 * k + i)
        value, bound = want(*ops, form, fa, fb)
        for out in OUTS.values():
            d = torch.full((m, n), float("nan"), dtype=out, device=DEV)
            call(*ops, d, form, fa, fb)
            R.check(d, value, bound)


@pytest.mark.parametrize("form", ["nk", "kn", "tiles"])
@pytest.mark.parametrize("fa,fb", list(itertools.product([0, 1], [0, 1])))
def test_formats(form, fa, fb):
    ops = operands(140, 272, 512, form, fa, fb, 5)
    d = torch.empty((140, 272), device=DEV)
    call(*ops, d, form, fa, fb)
    R.check(d, *want(*ops, form, fa, fb))


@pytest.mark.parametrize("m", [4, 150, 700])
@pytest.mark.parametrize("form", ["nk", "kn", "tiles"])
def test_special_codes(form, m):
    """NaN codes and E5M2 infinities reach exactly the outputs that fp32 arithmetic gives."""
    n, k, fa, fb = 300, 656, 1, 0
    a, sa, b, sb = operands(m, n, k, form, fa, fb, 11)
    a[1, 5], a[3, 600], a[2, 17] = 0x7F, 0x7C, 0xFC
    bt = b if form == "kn" else b.T
    bt[40, 9], bt[655, 299] = 0x7F, 0xFF
    bt[17, :] = 0x38  # the infinity of row 2 meets 1.0 everywhere ...
    bt[17, 30] = 0x00  # ... and a zero once
    d = torch.empty((m, n), device=DEV)
    call(a, sa, b, sb, d, form, fa, fb)
    value, bound = want(a, sa, b, sb, form, fa, fb)
    R.check(d, value, bound)


@pytest.mark.parametrize("form", ["nk", "kn", "tiles"])
@pytest.mark.parametrize("m,n,k", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (0, 0, 0), (300, 300, 0)])
def test_empty(form, m, n, k):
    d = torch.full((m, n), 3.0, device=DEV)
    call(*operands(m, n, k, form, 0, 0, 1), d, form, 0, 0)
    assert torch.equal(d, torch.zeros_like(d))
    d.fill_(3.0)
    call(*operands(m, n, k, form, 0, 0, 1), d, form, 0, 0, accumulate=True)
    assert (d == 3.0).all() or k > 0


@pytest.mark.parametrize("form", ["nk", "kn", "tiles"])
@pytest.mark.parametrize("m,n,k", [(3, 256, 512), (70, 257, 256), (300, 520, 384), (513, 640, 100)])
def test_accumulate(form, m, n, k):
    ops = operands(m, n, k, form, 1, 0, 21)
    value, bound = want(*ops, form, 1, 0)
    start = torch.randn((m, n), generator=gen(3), device=DEV) * value.abs().mean().float()
    d = start.clone()
    call(*ops, d, form, 1, 0, accumulate=True)
    R.check(d, value + start.double(), bound + 2.0 ** -24 * (value + start.double()).abs())


@pytest.mark.parametrize("off_a,off_b,off_d", [(1, 0, 0), (0, 3, 0), (0, 0, 1), (16, 16, 16), (5, 7, 3)])
@pytest.mark.parametrize("form", ["nk", "kn", "tiles"])
def test_unaligned_and_canaries(form, off_a, off_b, off_d):
    """Operands and output at odd addresses inside larger buffers; nothing outside D is written."""
    m, n, k = 150, 272, 400
    a, sa, b, sb = operands(m, n, k, form, 0, 0, 9)

    def at(t, off):
        buf = torch.full((t.numel() + 64,), 0x7F, dtype=torch.uint8, device=DEV)
        buf[off:off + t.numel()] = t.reshape(-1)
        return buf[off:off + t.numel()].view(t.shape)

    for out in OUTS.values():
        buf = torch.full((m * n + 256,), 77.0, dtype=out, device=DEV)
        d = buf[128 + off_d:128 + off_d + m * n].view(m, n)
        call(at(a, off_a), sa, at(b, off_b), sb, d, form, 0, 0)
        R.check(d, *want(a, sa, b, sb, form, 0, 0))
        assert (buf[:128 + off_d] == 77.0).all() and (buf[128 + off_d + m * n:] == 77.0).all()


def test_other_stream_and_repeat():
    """The same product on another stream and again is the same bits."""
    for m, n, k in [(8, 1024, 4096), (512, 1024, 2048)]:
        ops = operands(m, n, k, "nk", 0, 0, 2)
        d0, d1 = torch.empty((m, n), device=DEV), torch.empty((m, n), device=DEV)
        call(*ops, d0, "nk", 0, 0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        call(*ops, d1, "nk", 0, 0, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(d0, d1)
        for _ in range(5):
            call(*ops, d1, "nk", 0, 0)
            assert torch.equal(d0, d1)


def test_graph_capture():
    m, n, k = 40, 1024, 2048
    ops = operands(m, n, k, "nk", 0, 0, 2)
    d, big = torch.empty((m, n), device=DEV), torch.empty((512, n), device=DEV)
    ops2 = operands(512, n, k, "kn", 0, 0, 3)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call(*ops, d, "nk", 0, 0)
        call(*ops2, big, "kn", 0, 0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(*ops, d, "nk", 0, 0)
        call(*ops2, big, "kn", 0, 0)
    d.zero_(), big.zero_()
    g.replay()
    torch.cuda.synchronize()
    R.check(d, *want(*ops, "nk", 0, 0))
    R.check(big, *want(*ops2, "kn", 0, 0))


def test_output_offsets_beyond_32_bits():
    """More than 2^32 outputs: the last rows are where 32-bit offsets would wrap."""
    m, n, k = 70000, 65536, 32
    a, sa, b, sb = operands(m, n, k, "nk", 0, 0, 4)
    d = torch.zeros((m, n), dtype=torch.bfloat16, device=DEV)
    call(a, sa, b, sb, d, "nk", 0, 0)
    for rows in (slice(0, 130), slice(32000, 32100), slice(65500, 65600), slice(69990, 70000)):
        R.check(d[rows], *want(a[rows], sa[rows], b, sb, "nk", 0, 0))


# ------------------------------------------------------------------- grouped

GROUPS = {
    "one": [300],
    "two": [1, 299],
    "empty_first_last": [0, 130, 0, 0, 126, 44, 0],
    "all_empty": [0, 0, 0],
    "odd": [3, 0, 129, 1, 255, 77, 128, 256, 1],
    "tokens": [1, 0, 2, 1, 0, 0, 3, 1, 0, 1],
    "many": [(7 * i) % 11 for i in range(90)],
}


def ends_of(counts):
    return torch.tensor(counts, dtype=torch.int64, device=DEV).cumsum(0)


def grouped_want(counts, rows, a, sa, b, sb, form, fa, fb):
    n = b.shape[2 if form == "kn" else 1]
    value = torch.zeros((rows, n), dtype=torch.float64, device=DEV)
    bound, start = torch.zeros_like(value), 0
    for e, c in enumerate(counts):
        r = slice(start, start + c)
        if c:
            value[r], bound[r] = want(a[r], sa[r], b[e], sb[e], form, fa, fb)
        start += c
    return value, bound


@pytest.mark.parametrize("form", ["nk", "kn"])
@pytest.mark.parametrize("n,k", [(256, 512), (384, 1040), (130, 200), (1024, 256), (48, 1001)])
@pytest.mark.parametrize("kind", list(GROUPS))
def test_grouped(kind, n, k, form):
    counts = GROUPS[kind]
    for spare, (fa, fb), out in [(0, (0, 0), "bf16"), (70, (1, 0), "fp32")]:
        rows, e = sum(counts) + spare, len(counts)
        g = gen(n + k + rows)
        a, sa = R.finite_codes((rows, k), fa, g, DEV), R.scales((rows, blocks(k)), g, DEV)
        shape, sshape = ((e, k, n), (e, blocks(k), blocks(n))) if form == "kn" else ((e, n, k), (e, blocks(n), blocks(k)))
        b, sb = R.finite_codes(shape, fb, g, DEV), R.scales(sshape, g, DEV)
        if spare:  # rows of no group may hold anything
            a[sum(counts):] = 0x7F
        d = torch.full((rows, n), float("nan"), dtype=OUTS[out], device=DEV)
        fq.fp8_gemm_block_grouped(a, sa, b, sb, ends_of(counts), d, fa, fb, b_layout=fq.B_KN if form == "kn" else fq.B_NK)
        R.check(d, *grouped_want(counts, rows, a, sa, b, sb, form, fa, fb))


@pytest.mark.parametrize("form", ["nk", "kn"])
def test_grouped_neighbours_do_not_leak(form):
    """NaN codes of one expert's rows or weights stay out of every other expert's results,
    at tails of the contraction (k = 200) where a block of one expert ends inside a tile."""
    counts, n, k = [100, 28, 0, 150], 130, 208
    rows, e, g = sum(counts), len(counts), gen(6)
    a, sa = R.finite_codes((rows, k), 0, g, DEV), R.scales((rows, blocks(k)), g, DEV)
    shape, sshape = ((e, k, n), (e, blocks(k), blocks(n))) if form == "kn" else ((e, n, k), (e, blocks(n), blocks(k)))
    b, sb = R.finite_codes(shape, 0, g, DEV), R.scales(sshape, g, DEV)
    a[100:128] = 0x7F
    b[2], b[1] = 0x7F, 0x7F
    d = torch.empty((rows, n), device=DEV)
    fq.fp8_gemm_block_grouped(a, sa, b, sb, ends_of(counts), d, b_layout=fq.B_KN if form == "kn" else fq.B_NK)
    R.check(d, *grouped_want(counts, rows, a, sa, b, sb, form, 0, 0))
    assert d[:100].isfinite().all() and d[128:].isfinite().all() and d[100:128].isnan().all()


@pytest.mark.parametrize("bad,counts", [([-5, 40, 20, 500], [0, 40, 0, 60]), ([200, 50, 100, 100], [100, 0, 0, 0]),
                                        ([10, 2 ** 40, 3, 50], [10, 90, 0, 0])])
def test_group_ends_are_clamped(bad, counts):
    rows, n, k, e = 100, 256, 256, 4
    g = gen(8)
    a, sa = R.finite_codes((rows, k), 0, g, DEV), R.scales((rows, 2), g, DEV)
    b, sb = R.finite_codes((e, n, k), 0, g, DEV), R.scales((e, 2, 2), g, DEV)
    d = torch.empty((rows, n), device=DEV)
    ends = torch.tensor(bad, dtype=torch.int64, device=DEV)
    fq.fp8_gemm_block_grouped(a, sa, b, sb, ends, d)
    R.check(d, *grouped_want(counts, rows, a, sa, b, sb, "nk", 0, 0))
    at, st, bt, ut = (R.finite_codes((n, rows), 0, g, DEV), R.scales((n, 1), g, DEV),
                      R.finite_codes((k, rows), 0, g, DEV), R.scales((k, 1), g, DEV))
    dw = torch.empty((e, n, k), device=DEV)
    fq.fp8_gemm_block_grouped_wgrad(at, st, bt, ut, ends, dw)
    check_wgrad(dw, counts, at, st, bt, ut, 0, 0)


def test_grouped_weight_offsets_beyond_32_bits():
    e, n, k = 40, 16384, 8192  # 5.4e9 bytes of weights
    counts = [2] * e
    g = gen(4)
    a, sa = R.finite_codes((2 * e, k), 0, g, DEV), R.scales((2 * e, blocks(k)), g, DEV)
    b = torch.randint(0, 0x70, (e, n, k), generator=g, device=DEV, dtype=torch.uint8)
    sb = R.scales((e, blocks(n), blocks(k)), g, DEV)
    d = torch.empty((2 * e, n), device=DEV)
    fq.fp8_gemm_block_grouped(a, sa, b, sb, ends_of(counts), d)
    for i in (0, 20, 31, 32, 39):
        cols = slice(n - 256, n)
        r = slice(2 * i, 2 * i + 2)
        R.check(d[r, cols], *want(a[r], sa[r], b[i, cols], sb[i, -2:], "nk", 0, 0))


# ---------------------------------------------------------- grouped wgrad

def check_wgrad(d, counts, a, sa, b, sb, fa, fb, start_value=None):
    av, bv, start = R.values(a, sa, fa, 1), R.values(b, sb, fb, 1), 0
    blocks_all = blocks(a.shape[1])
    for e, c in enumerate(counts):
        value, bound = R.product(av[:, start:start + c], bv[:, start:start + c])
        # a group that is not aligned to 128 touches one block more than its length says
        bound = bound * (128 + blocks_all + 5) / (128 + 4)
        if start_value is not None:
            value = value + start_value[e].double()
            bound = bound + 2.0 ** -24 * value.abs()
        R.check(d[e], value, bound)
        start += c


WGRAD = dict(GROUPS, aligned=[128, 256, 0, 384], aligned_16=[16, 112, 48, 0, 320, 64], cut=[100, 28, 128, 200, 56],
             inside=[10, 20, 30, 40, 28])


@pytest.mark.parametrize("m,n", [(128, 256), (256, 384), (130, 70), (300, 520), (1, 33)])
@pytest.mark.parametrize("kind", list(WGRAD))
def test_grouped_wgrad(kind, m, n):
    counts = WGRAD[kind]
    for spare, (fa, fb), out in [(0, (1, 0), "fp32"), (37, (0, 0), "bf16"), (-sum(counts) % 16 + 16, (0, 1), "fp32")]:
        rows, e = sum(counts) + spare, len(counts)
        g = gen(m + n + rows)
        a, sa = R.finite_codes((m, rows), fa, g, DEV), R.scales((m, blocks(rows)), g, DEV)
        b, sb = R.finite_codes((n, rows), fb, g, DEV), R.scales((n, blocks(rows)), g, DEV)
        if spare:
            a[:, sum(counts):], b[:, sum(counts):] = 0x7F, 0x7F
        d = torch.full((e, m, n), float("nan"), dtype=OUTS[out], device=DEV)
        fq.fp8_gemm_block_grouped_wgrad(a, sa, b, sb, ends_of(counts), d, fa, fb)
        check_wgrad(d, counts, a, sa, b, sb, fa, fb)


def test_grouped_wgrad_neighbours_do_not_leak():
    """A 128-row scale tile shared by two experts: the other's NaN codes never reach the sum."""
    counts, m, n = [100, 28, 5, 59, 192], 256, 272
    rows, g = sum(counts), gen(3)
    a, sa = R.finite_codes((m, rows), 0, g, DEV), R.scales((m, blocks(rows)), g, DEV)
    b, sb = R.finite_codes((n, rows), 0, g, DEV), R.scales((n, blocks(rows)), g, DEV)
    a[:, 100:128], b[:, 128:133] = 0x7F, 0x7F
    d = torch.empty((len(counts), m, n), device=DEV)
    fq.fp8_gemm_block_grouped_wgrad(a, sa, b, sb, ends_of(counts), d)
    check_wgrad(d, counts, a, sa, b, sb, 0, 0)
    assert d[0].isfinite().all() and d[3].isfinite().all() and d[4].isfinite().all()


@pytest.mark.parametrize("kind", ["odd", "aligned", "empty_first_last"])
def test_grouped_wgrad_accumulates(kind):
    counts, m, n = WGRAD[kind], 256, 300
    rows, g = sum(counts), gen(5)
    a, sa = R.finite_codes((m, rows), 1, g, DEV), R.scales((m, blocks(rows)), g, DEV)
    b, sb = R.finite_codes((n, rows), 0, g, DEV), R.scales((n, blocks(rows)), g, DEV)
    start = torch.randn((len(counts), m, n), generator=g, device=DEV) * 100
    d = start.clone()
    fq.fp8_gemm_block_grouped_wgrad(a, sa, b, sb, ends_of(counts), d, 1, 0, accumulate=True)
    check_wgrad(d, counts, a, sa, b, sb, 1, 0, start)


# -------------------------------------------------- as gradients of a layer

def test_products_are_the_gradients_of_the_forward_product():
    """The three products over one layer's own quantized operands: dgrad and wgrad against
    central differences of the forward product's 64-bit form with the same operands."""
    t, out, inn = 160, 256, 384
    g = gen(13)
    x = torch.randn((t, inn), generator=g, device=DEV).bfloat16()
    w = (torch.randn((out, inn), generator=g, device=DEV) * 0.05).bfloat16()
    dy = torch.randn((t, out), generator=g, device=DEV).bfloat16()

    def block_ct(v):
        r, c = v.shape
        qr, qc = torch.empty((r, c), dtype=torch.uint8, device=DEV), torch.empty((c, r), dtype=torch.uint8, device=DEV)
        sr, sc = torch.empty((r, blocks(c)), device=DEV), torch.empty((c, blocks(r)), device=DEV)
        fq.fp8_quantize_block_cast_transpose(v, fq.E4M3, qr, sr, qc, sc)
        return qr, sr, qc, sc

    xr, xsr, xc, xsc = block_ct(x)
    gr, gsr, gc, gsc = block_ct(dy)
    qw, sw = torch.empty((out, inn), dtype=torch.uint8, device=DEV), torch.empty((blocks(out), blocks(inn)), device=DEV)
    fq.fp8_quantize_block(w, 128, 128, fq.E4M3, qw, sw)
    y = torch.empty((t, out), device=DEV)
    dx, dw = torch.empty((t, inn), device=DEV), torch.empty((out, inn), device=DEV)
    fq.fp8_gemm_block(xr, xsr, qw, sw, y)
    fq.fp8_gemm_block(gr, gsr, qw, sw, dx, b_layout=fq.B_KN)
    fq.fp8_gemm_block(gc, gsc, xc, xsc, dw, b_block_rows=1)
    wv = R.values(qw, sw, 0, 128)
    R.check(y, *R.product(R.values(xr, xsr, 0, 1), wv))
    # loss = sum(dY * Y), linear in X and in W: differences are exact up to rounding
    gv, xv = R.values(gr, gsr, 0, 1), R.values(xr, xsr, 0, 1)
    gv2, xv2 = R.values(gc, gsc, 0, 1).T, R.values(xc, xsc, 0, 1).T
    _, bound_x = R.product(gv, wv.T)
    _, bound_w = R.product(gv2.T, xv2.T)
    h = 0.5
    for i, j in [(0, 0), (17, 200), (159, 383)]:
        e = torch.zeros_like(xv)
        e[i, j] = h
        diff = ((gv * ((xv + e) @ wv.T)).sum() - (gv * ((xv - e) @ wv.T)).sum()) / (2 * h)
        assert abs(dx[i, j].double() - diff) <= bound_x[i, j] + 1e-8 * (gv.abs() @ wv.abs())[i, j] * t
    for i, j in [(0, 0), (100, 300), (255, 383)]:
        e = torch.zeros_like(wv)
        e[i, j] = h
        diff = ((gv2 * (xv2 @ (wv + e).T)).sum() - (gv2 * (xv2 @ (wv - e).T)).sum()) / (2 * h)
        assert abs(dw[i, j].double() - diff) <= bound_w[i, j] + 1e-8 * (gv2.abs().T @ xv2.abs())[i, j] * out


def test_no_wait_gave_up():
    """Every product above ended by itself: no bounded wait reached its limit."""
    assert fq.wait_timeouts() == 0


def test_scratch_of_odd_operands_is_kept_and_released():
    """Odd rows are copied into the stream's scratch: it grows, serves smaller calls, and can be released."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for m, n, k in [(20, 256, 333), (300, 520, 1001), (20, 256, 333)]:
            ops = operands(m, n, k, "nk", 0, 0, m + k)
            d = torch.empty((m, n), device=DEV)
            call(*ops, d, "nk", 0, 0)
            R.check(d, *want(*ops, "nk", 0, 0))
        fq.release_stream_workspace(s)
        ops = operands(40, 130, 77, "kn", 0, 0, 1)
        d = torch.empty((40, 130), device=DEV)
        call(*ops, d, "kn", 0, 0)
        R.check(d, *want(*ops, "kn", 0, 0))
        fq.release_stream_workspace(s)
