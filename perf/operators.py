"""Measured cases of the block-scaled FP8 products and of gradient clipping.

Three operators, each with a plain form in 32 bits (elementary torch
operations) and the library's own calls:

  linear   fp8_gemm_block                 D[m, n] = sum_k A[m, k] B[n, k] over FP8 codes with one
                                          scale per 1 x 128 tile of A and per 128 x 128 block (or
                                          1 x 128 tile) of B
  experts  fp8_gemm_block_grouped         the same product for rows sorted by expert, ragged sizes
           fp8_gemm_block_grouped_wgrad   one weight gradient per expert, summed over its rows
  clip     fp8_grad_clip_grouped          global gradient norm over many tensors and clipping

`own` selects the library's calls; the tree's package is imported only then.
"""
import math
import random

import numpy as np
import torch

own = False

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
OUT = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128
EPS = 1e-6  # added to the norm before the division, as training loops do


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # The smallest call: a few tokens through a small projection, where launch latency counts.
        dict(name="linear-latency", op="linear", dir="forward", m=3, n=1024, k=1024, fmt_a="e4m3", out="bf16"),
        # Serving one token: the down projection's weight is read once, nothing else counts.
        dict(name="linear-token", op="linear", dir="forward", m=1, n=7168, k=18432, fmt_a="e4m3", out="bf16"),
        # Serving a batch of single tokens.
        dict(name="linear-batch", op="linear", dir="forward", m=48, n=14336, k=4096, fmt_a="e4m3", out="bf16"),
        # Training or prefill, forward, with a ragged number of tokens.
        dict(name="linear-forward", op="linear", dir="forward", m=4001, n=7168, k=18432, fmt_a="e4m3", out="bf16"),
        # The largest: gradient of a layer's input, E5M2 gradients times the weight as it is stored.
        dict(name="linear-dgrad", op="linear", dir="dgrad", m=16384, n=18432, k=7168, fmt_a="e5m2", out="bf16"),
        # Gradient of a layer's weight: both operands in 1 x 128 tiles along the tokens, FP32 main gradient.
        dict(name="linear-wgrad", op="linear", dir="wgrad", m=4096, n=14336, k=8192, fmt_a="e5m2", out="fp32"),
        # Serving a mixture of experts: a couple of tokens for each, some experts idle.
        dict(name="experts-decode", op="experts", dir="forward", rows=96, experts=64, n=2048, k=7168, skew=0.5,
             idle=16, spare=0, fmt_a="e4m3", out="bf16"),
        # Training or prefill through all experts; uneven, two idle, some rows of the buffer unused.
        dict(name="experts-forward", op="experts", dir="forward", rows=16384, experts=32, n=4096, k=7168, skew=0.7,
             idle=2, spare=100, fmt_a="e4m3", out="bf16"),
        # Gradient of the experts' inputs.
        dict(name="experts-dgrad", op="experts", dir="dgrad", rows=8191, experts=16, n=7168, k=2048, skew=0.5,
             idle=1, spare=0, fmt_a="e5m2", out="bf16"),
        # Gradients of the experts' weights; an odd number of rows, so no operand row is 16-byte aligned.
        dict(name="experts-wgrad", op="experts", dir="wgrad", rows=8195, experts=16, n=7168, k=2048, skew=0.5,
             idle=1, spare=0, fmt_a="e5m2", out="fp32"),
        # Clipping a small model's gradients: many small tensors, latency counts.
        dict(name="clip-small", op="clip", tensors=64, elements=1 << 20, sizes="ragged", src="mixed", out="fp32",
             max_norm=0.5),
        # Clipping a large model's BF16 gradients into the optimizer's FP32 main gradients.
        dict(name="clip-large", op="clip", tensors=290, elements=1500000000, sizes="ragged", src="bf16", out="fp32",
             max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size over the logarithm of [lo, hi]: a multiple of 128, of 16, or any number."""
    v, kind = _log(rng, lo, hi), rng.random()
    step = 128 if kind < 0.5 else 16 if kind < 0.75 else 1
    return max(1, v // step * step or v)


def draw(rng):
    op = rng.choice(["linear", "linear", "experts", "experts", "clip"])
    if op == "clip":
        return dict(op="clip", tensors=_log(rng, 1, 400), elements=_log(rng, 1 << 14, 1 << 29),
                    sizes=rng.choice(["even", "ragged"]), src=rng.choice(["bf16", "fp32", "mixed"]),
                    out=rng.choice(["bf16", "fp32"]), max_norm=rng.choice([0.01, 0.1, 1.0, 1e6]))
    direction = rng.choice(["forward", "dgrad", "wgrad"])
    fmt_a = "e4m3" if direction == "forward" else rng.choice(["e4m3", "e5m2"])
    out = "fp32" if direction == "wgrad" else rng.choice(["bf16", "bf16", "fp32"])
    if op == "linear":
        m, n, k = _size(rng, 1, 8192), _size(rng, 256, 16384), _size(rng, 256, 16384)
        if direction == "wgrad":
            m, k = _size(rng, 256, 8192), _size(rng, 64, 16384)
        while m * n * k > 5e11:
            m = max(1, m // 2)
        return dict(op=op, dir=direction, m=m, n=n, k=k, fmt_a=fmt_a, out=out)
    experts, rows = _log(rng, 2, 64), _size(rng, 16, 16384)
    n, k = _size(rng, 256, 4096), _size(rng, 256, 7168)
    while experts * n * k > 5e8:
        experts = max(2, experts // 2)
    return dict(op=op, dir=direction, rows=rows, experts=experts, n=n, k=k, skew=round(rng.uniform(0.0, 1.0), 2),
                idle=rng.randrange(0, max(1, experts // 4)), spare=rng.choice([0, 0, rng.randrange(1, 200)]),
                fmt_a=fmt_a, out=out)


def _counts(case):
    """Rows of each expert: from the case alone (the seed only permutes them), `idle` of them without any."""
    rng = np.random.RandomState(case["rows"] * 131 + case["experts"])
    busy = max(1, case["experts"] - case["idle"])
    p = np.exp(rng.standard_normal(busy) * case["skew"])
    total = max(0, case["rows"] - case["spare"])
    counts = np.zeros(case["experts"], np.int64)
    counts[:busy] = np.floor(total * p / p.sum()).astype(np.int64)
    counts[int(np.argmax(counts[:busy]))] += total - counts.sum()
    return counts


def _sizes(case):
    """Elements of each gradient tensor: equal shares, or many vectors beside a few matrices."""
    c, total = case["tensors"], case["elements"]
    if case["sizes"] == "even":
        w = np.ones(c)
    else:
        rng = np.random.RandomState(c * 17 + total % 1009)
        w = np.exp(rng.uniform(np.log(1e-4), 0.0, c))
    s = np.maximum(1, np.floor(total * w / w.sum())).astype(np.int64)
    return [int(v) for v in s]


def _sources(case):
    return ["fp32" if case["src"] == "fp32" or (case["src"] == "mixed" and i % 3 == 2) else "bf16"
            for i in range(case["tensors"])]


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    size = 2 if case["out"] == "bf16" else 4
    if case["op"] == "clip":
        s = _sizes(case)
        src = sum(v * (4 if t == "fp32" else 2) for v, t in zip(s, _sources(case)))
        # one square and add, one product per element; the input once, the output once
        return {"bytes": src + sum(s) * size + 4, "flops": 3 * sum(s)}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        sb = 4 * _blocks(k) * (n if case["dir"] == "wgrad" else _blocks(n))
        return {"bytes": m * k + 4 * m * _blocks(k) + n * k + sb + m * n * size, "flops": 2 * m * n * k}
    t, n, k = case["rows"], case["n"], case["k"]
    counts = _counts(case)
    used, busy = int(counts.sum()), int((counts > 0).sum())
    if case["dir"] == "wgrad":  # [k, rows] and [n, rows] codes, a gradient for every expert
        return {"bytes": used * (n + k) + 4 * _blocks(used) * (n + k) + case["experts"] * (n * k * size + 8),
                "flops": 2 * used * n * k}
    weight = n * k + 4 * _blocks(n) * _blocks(k)
    return {"bytes": used * (k + 4 * _blocks(k)) + busy * weight + t * n * size + 8 * case["experts"],
            "flops": 2 * used * n * k}


# ----------------------------------------------------------------- the inputs

def _codes(x, amax, fmt):
    """FP8 codes of x scaled to its block maxima, and the dequantization factors."""
    dtype, top = FP8[fmt]
    scale = torch.where(amax > 0, top / amax, torch.ones_like(amax))
    return scale, (1.0 / scale), dtype, top


def _quantize_rows(x, fmt):
    """1 x 128 tiles along the last axis: uint8 codes and float32 factors."""
    r, c = x.shape
    p = torch.nn.functional.pad(x, (0, _blocks(c) * BLOCK - c)).view(r, _blocks(c), BLOCK)
    scale, inv, dtype, top = _codes(p, p.abs().amax(-1), fmt)
    q = (p * scale[..., None]).clamp_(-top, top).to(dtype).view(torch.uint8).view(r, -1)[:, :c].contiguous()
    return q, inv.contiguous()


def _quantize_blocks(x, fmt):
    """128 x 128 blocks of the last two axes."""
    e, r, c = x.shape
    p = torch.nn.functional.pad(x, (0, _blocks(c) * BLOCK - c, 0, _blocks(r) * BLOCK - r))
    p = p.view(e, _blocks(r), BLOCK, _blocks(c), BLOCK)
    scale, inv, dtype, top = _codes(p, p.abs().amax((2, 4)), fmt)
    q = (p * scale[:, :, None, :, None]).clamp_(-top, top).to(dtype).view(torch.uint8)
    return q.view(e, _blocks(r) * BLOCK, -1)[:, :r, :c].contiguous(), inv.contiguous()


def _rows(gen, r, c, std):
    """Activations or gradients: normal values whose magnitude varies from tile to tile."""
    tile = torch.randn(r, _blocks(c), generator=gen, device="cuda").exp_().repeat_interleave(BLOCK, 1)[:, :c]
    return torch.randn(r, c, generator=gen, device="cuda").mul_(std).mul_(tile)


def _weights(gen, e, r, c):
    block = torch.randn(e, _blocks(r), _blocks(c), generator=gen, device="cuda").mul_(0.3).exp_()
    x = torch.randn(e, _blocks(r), BLOCK, _blocks(c), BLOCK, generator=gen, device="cuda").mul_(0.02)
    return x.mul_(block[:, :, None, :, None]).view(e, _blocks(r) * BLOCK, -1)[:, :r, :c]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "clip":
        return _prepare_clip(case, gen)
    s = {"case": case}
    out = OUT[case["out"]]
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = _quantize_rows(_rows(gen, m, k, 1.0), case["fmt_a"])
        if case["dir"] == "wgrad":
            s["b"], s["sb"] = _quantize_rows(_rows(gen, n, k, 1.0), "e4m3")
        else:
            shape = (n, k) if case["dir"] == "forward" else (k, n)
            b, sb = _quantize_blocks(_weights(gen, 1, *shape), "e4m3")
            s["b"], s["sb"] = b[0], sb[0]
        s["d"] = torch.empty(m, n, dtype=out, device="cuda")
        return s
    t, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
    counts = np.random.RandomState(int(seed) % (1 << 31)).permutation(_counts(case))
    s["ends"] = torch.from_numpy(np.cumsum(counts)).to("cuda")
    s["most"] = int(counts.max())  # the capacity that a padded layout needs
    if case["dir"] == "wgrad":
        s["a"], s["sa"] = _quantize_rows(_rows(gen, k, t, 1.0), case["fmt_a"])
        s["b"], s["sb"] = _quantize_rows(_rows(gen, n, t, 1.0), "e4m3")
        s["d"] = torch.empty(e, k, n, dtype=out, device="cuda")
        return s
    s["a"], s["sa"] = _quantize_rows(_rows(gen, t, k, 1.0), case["fmt_a"])
    s["b"], s["sb"] = _quantize_blocks(_weights(gen, e, *((n, k) if case["dir"] == "forward" else (k, n))), "e4m3")
    s["d"] = torch.empty(t, n, dtype=out, device="cuda")
    return s


def _prepare_clip(case, gen):
    """Gradient tensors, and views of one flat buffer for the clipped ones, each starting at a multiple of 64 elements."""
    sizes, s = _sizes(case), {"case": case}
    s["xs"] = [(torch.randn(v, generator=gen, device="cuda") * 1e-3).to(OUT[t]) for v, t in zip(sizes, _sources(case))]
    starts = np.concatenate([[0], np.cumsum([-(-v // 64) * 64 for v in sizes])])
    s["flat"] = torch.zeros(int(starts[-1]), dtype=OUT[case["out"]], device="cuda")
    s["ys"] = [s["flat"][a:a + v] for a, v in zip(starts.tolist(), sizes)]
    s["gaps"] = [torch.zeros(-v % 64, device="cuda") for v in sizes]
    s["norm"] = torch.empty(1, device="cuda")
    return s


# ------------------------------------------------------------- one pass each

def run(s):
    case = s["case"]
    if case["op"] == "clip":
        return _clip_own(s) if own else _clip_plain(s)
    return _product_own(s) if own else _product_plain(s)


def _product_own(s):
    import fp8_scaled_quantization_gb300 as fq
    case = s["case"]
    fmt_a = fq.E4M3 if case["fmt_a"] == "e4m3" else fq.E5M2
    layout = fq.B_KN if case["dir"] == "dgrad" else fq.B_NK
    if case["op"] == "linear":
        fq.fp8_gemm_block(s["a"], s["sa"], s["b"], s["sb"], s["d"], fmt_a, fq.E4M3, b_layout=layout,
                          b_block_rows=1 if case["dir"] == "wgrad" else BLOCK)
    elif case["dir"] == "wgrad":
        fq.fp8_gemm_block_grouped_wgrad(s["a"], s["sa"], s["b"], s["sb"], s["ends"], s["d"], fmt_a, fq.E4M3)
    else:
        fq.fp8_gemm_block_grouped(s["a"], s["sa"], s["b"], s["sb"], s["ends"], s["d"], fmt_a, fq.E4M3,
                                  b_layout=layout)
    return s["d"]


def _rows32(q, inv, fmt):
    c = q.shape[-1]
    return q.view(FP8[fmt][0]).float() * inv.repeat_interleave(BLOCK, -1)[..., :c]


def _blocks32(q, inv):
    r, c = q.shape[-2:]
    f = inv.repeat_interleave(BLOCK, -1)[..., :c].repeat_interleave(BLOCK, -2)[..., :r, :]
    return q.view(FP8["e4m3"][0]).float() * f


def _product_plain(s):
    case = s["case"]
    a = _rows32(s["a"], s["sa"], case["fmt_a"])
    b = _rows32(s["b"], s["sb"], "e4m3") if case["dir"] == "wgrad" else _blocks32(s["b"], s["sb"])
    if case["op"] == "linear":
        return (a @ (b if case["dir"] == "dgrad" else b.T)).to(s["d"].dtype)
    # every expert's rows in a padded block of its own, one batched product, rows taken back
    t, e, most = case["rows"], case["experts"], s["most"]
    row = torch.arange(t, device="cuda")
    group = torch.searchsorted(s["ends"], row, right=True)
    first = torch.cat([s["ends"].new_zeros(1), s["ends"]])[group]
    slot = torch.where(group < e, group * most + row - first, e * most)
    if case["dir"] == "wgrad":
        pa, pb = (torch.zeros(e * most + 1, x.shape[0], device="cuda") for x in (a, b))
        pa[slot], pb[slot] = a.T, b.T
        pa, pb = (x[:e * most].view(e, most, -1) for x in (pa, pb))
        return torch.bmm(pa.transpose(1, 2), pb).to(s["d"].dtype)
    pa = torch.zeros(e * most + 1, a.shape[1], device="cuda")
    pa[slot] = a
    d = torch.bmm(pa[:e * most].view(e, most, -1), b if case["dir"] == "dgrad" else b.transpose(1, 2))
    d = torch.cat([d.view(e * most, -1), d.new_zeros(1, d.shape[2])])
    return d[slot].to(s["d"].dtype)


def _clip_own(s):
    import fp8_scaled_quantization_gb300 as fq
    fq.fp8_grad_clip_grouped(s["xs"], s["case"]["max_norm"], s["norm"], ys=s["ys"], eps=EPS)
    return {"norm": s["norm"], "clipped": s["flat"]}


def _clip_plain(s):
    flat = torch.cat([v for x, gap in zip(s["xs"], s["gaps"]) for v in (x.float(), gap)])
    norm = (flat * flat).sum().sqrt()
    factor = (s["case"]["max_norm"] / (norm + EPS)).clamp(max=1.0)
    return {"norm": norm.reshape(1), "clipped": (flat * factor).to(s["flat"].dtype)}


# --------------------------------------------------------- the same in 64 bits

def _decoded(fmt):
    """The 256 values of a format, from its definition: sign, exponent and fraction fields."""
    e_bits, bias = (4, 7) if fmt == "e4m3" else (5, 15)
    m_bits, values = 7 - e_bits, []
    for code in range(256):
        e, f = (code >> m_bits) & ((1 << e_bits) - 1), code & ((1 << m_bits) - 1)
        v = (1 + f / 2 ** m_bits) * 2.0 ** (e - bias) if e else f / 2 ** m_bits * 2.0 ** (1 - bias)
        if fmt == "e4m3" and e == 15 and f == 7:
            v = math.nan
        if fmt == "e5m2" and e == 31:
            v = math.nan if f else math.inf
        values.append(-v if code & 128 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _wide(q, inv, fmt, block_rows):
    """Dequantized values in 64 bits, scales indexed by row and column block."""
    r, c = q.shape
    at = torch.arange(r, device="cuda")[:, None] // block_rows, torch.arange(c, device="cuda")[None, :] // BLOCK
    return _decoded(fmt)[q.long()] * inv.double()[at]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        square = sum((x.double() ** 2).sum() for x in s["xs"])
        norm = square.sqrt()
        factor = min(1.0, case["max_norm"] / (float(norm) + EPS))
        flat, at = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda"), 0
        for x in s["xs"]:
            flat[at:at + x.numel()] = x.double() * factor
            at += -(-x.numel() // 64) * 64
        return {"norm": norm.reshape(1), "clipped": flat}
    if case["op"] == "linear":
        a = _wide(s["a"], s["sa"], case["fmt_a"], 1)
        b = _wide(s["b"], s["sb"], "e4m3", 1 if case["dir"] == "wgrad" else BLOCK)
        return a @ (b if case["dir"] == "dgrad" else b.T)
    d, start = torch.zeros(s["d"].shape, dtype=torch.float64, device="cuda"), 0
    if case["dir"] == "wgrad":
        a, b = _wide(s["a"], s["sa"], case["fmt_a"], 1), _wide(s["b"], s["sb"], "e4m3", 1)
    for e, end in enumerate(s["ends"].tolist()):
        if end > start and case["dir"] == "wgrad":
            d[e] = a[:, start:end] @ b[:, start:end].T
        elif end > start:
            w = _wide(s["b"][e], s["sb"][e], "e4m3", BLOCK)
            x = _wide(s["a"][start:end], s["sa"][start:end], case["fmt_a"], 1)
            d[start:end] = x @ (w if case["dir"] == "dgrad" else w.T)
        start = end
    return d


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
