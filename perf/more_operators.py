"""Measured cases of the gated feed-forward block in block-scaled FP8, with its 8-bit checkpoint.

Three operators, each with a plain form in 32 bits (elementary torch
operations) and the library's own calls:

  gated     fp8_gemm_block_gated           h = act(X Wg^T) * (X Wu^T) over FP8 codes, both projections,
                                           the activation and the product in one call; h comes as FP8
                                           codes with one factor per 1 x 128 tile, and so does, where it
                                           is asked for, the checkpoint: both projections
  experts   fp8_gemm_block_gated_grouped   the same for rows sorted by expert, ragged sizes
  backward  fp8_gated_block_backward       from the gradient of h and the checkpoint: the gradients of
                                           both projections as FP8 codes, along their rows and
                                           transposed, and h transposed

What is held in 8 bits is returned as float8 tensors (the codes' values) beside
their factors.  `own` selects the library's calls; the tree's package is
imported only then.
"""
import math
import random

import numpy as np
import torch

own = False

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
OUT = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128
GELU_C, GELU_CUBE = math.sqrt(2.0 / math.pi), 0.044715  # of the tanh form


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # The smallest call: a few tokens through a small block, where launch latency counts.
        dict(name="gated-latency", op="gated", m=3, n=1024, k=1024, act="silu", keep=False),
        # Serving one token: both weights are read once, nothing else counts.
        dict(name="gated-token", op="gated", m=1, n=18432, k=7168, act="silu", keep=False),
        # Serving a batch of single tokens.
        dict(name="gated-batch", op="gated", m=48, n=14336, k=4096, act="silu", keep=False),
        # Sizes that no tile divides, operand and output rows that are not 16-byte aligned.
        dict(name="gated-odd", op="gated", m=777, n=4100, k=1032, act="gelu", keep=True),
        # Training or prefill: a ragged number of tokens, with the checkpoint for the backward pass.
        dict(name="gated-forward", op="gated", m=4001, n=18432, k=7168, act="silu", keep=True),
        # Serving a mixture of experts: a couple of tokens for each, some experts idle.
        dict(name="experts-decode", op="experts", rows=96, experts=64, n=2048, k=7168, skew=0.5, idle=16, spare=0,
             act="silu", keep=False),
        # Training all experts: uneven, two idle, some rows of the buffer unused.
        dict(name="experts-forward", op="experts", rows=16384, experts=32, n=2048, k=7168, skew=0.7, idle=2,
             spare=100, act="silu", keep=True),
        # The backward pass of a few tokens: latency counts.
        dict(name="backward-small", op="backward", rows=17, n=1024, act="silu", grad="bf16", fmt="e4m3"),
        # A training step's rows through a layer of 14336.
        dict(name="backward-train", op="backward", rows=4096, n=14336, act="silu", grad="bf16", fmt="e4m3"),
        # All experts' rows at once, an odd number: no transposed row is aligned; fp32 gradients.
        dict(name="backward-odd", op="backward", rows=8195, n=2048, act="gelu", grad="fp32", fmt="e4m3"),
        # The largest: a long batch, gradients in E5M2.
        dict(name="backward-large", op="backward", rows=16384, n=18432, act="silu", grad="bf16", fmt="e5m2"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size over the logarithm of [lo, hi]: a multiple of 128, of 16, or any number."""
    v, kind = _log(rng, lo, hi), rng.random()
    step = 128 if kind < 0.5 else 16 if kind < 0.75 else 1
    return max(1, v // step * step or v)


def draw(rng):
    op, act = rng.choice(["gated", "gated", "experts", "backward", "backward"]), rng.choice(["silu", "silu", "gelu"])
    if op == "backward":
        return dict(op=op, rows=_size(rng, 1, 16384), n=_size(rng, 128, 18432), act=act,
                    grad=rng.choice(["bf16", "bf16", "fp32"]), fmt=rng.choice(["e4m3", "e5m2"]))
    keep = rng.random() < 0.5
    if op == "gated":
        m, n, k = _size(rng, 1, 8192), _size(rng, 128, 18432), _size(rng, 128, 8192)
        while m * n * k > 4e11:
            m = max(1, m // 2)
        return dict(op=op, m=m, n=n, k=k, act=act, keep=keep)
    experts, rows = _log(rng, 2, 64), _size(rng, 16, 16384)
    n, k = _size(rng, 128, 4096), _size(rng, 128, 7168)
    while experts * n * k > 4e8:
        experts = max(2, experts // 2)
    return dict(op=op, rows=rows, experts=experts, n=n, k=k, skew=round(rng.uniform(0.0, 1.0), 2),
                idle=rng.randrange(0, max(1, experts // 4)), spare=rng.choice([0, 0, rng.randrange(1, 200)]),
                act=act, keep=keep)


def _counts(case):
    """Rows of each expert: from the case alone (the seed only permutes them), `idle` of them without any."""
    rng = np.random.RandomState(case["rows"] * 137 + case["experts"])
    busy = max(1, case["experts"] - case["idle"])
    p = np.exp(rng.standard_normal(busy) * case["skew"])
    total = max(0, case["rows"] - case["spare"])
    counts = np.zeros(case["experts"], np.int64)
    counts[:busy] = np.floor(total * p / p.sum()).astype(np.int64)
    counts[int(np.argmax(counts[:busy]))] += total - counts.sum()
    return counts


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    n = case["n"]
    if case["op"] == "backward":
        rows = case["rows"]
        grad = 2 if case["grad"] == "bf16" else 4
        factors = 4 * (rows * 4 * _blocks(n) + 3 * n * _blocks(rows))
        # gradient and checkpoint in; both gradients twice and h once out; per element the
        # decoding, sigmoid and derivative, products, maxima and scaling
        return {"bytes": rows * n * (grad + 2 + 2 + 2 + 1) + factors, "flops": 30 * rows * n}
    k, kept = case["k"], 2 if case["keep"] else 0
    if case["op"] == "gated":
        rows = used = case["m"]
        busy, ends = 1, 0
    else:
        counts = _counts(case)
        rows, used, busy, ends = case["rows"], int(counts.sum()), int((counts > 0).sum()), 8 * case["experts"]
    weights = busy * 2 * (n * k + 4 * _blocks(n) * _blocks(k))
    return {"bytes": used * (k + 4 * _blocks(k)) + weights + rows * (1 + kept) * (n + 4 * _blocks(n)) + ends,
            "flops": used * n * (4 * k + 10)}


# ----------------------------------------------------------------- the inputs

def _tiles(x, top, dtype):
    """1 x 128 tiles along the last axis: float8 codes and float32 factors (1 for tiles of zeros)."""
    c = x.shape[-1]
    p = torch.nn.functional.pad(x, (0, _blocks(c) * BLOCK - c)).view(*x.shape[:-1], _blocks(c), BLOCK)
    amax = p.abs().amax(-1)
    scale = torch.where(amax > 0, top / amax, torch.ones_like(amax))
    q = (p * scale[..., None]).clamp_(-top, top).to(dtype).view(*x.shape[:-1], -1)[..., :c].contiguous()
    return q, (1.0 / scale).contiguous()


def _rows(gen, r, c, std):
    """Values whose magnitude varies from tile to tile."""
    tile = torch.randn(r, _blocks(c), generator=gen, device="cuda").mul_(0.5).exp_()
    return torch.randn(r, c, generator=gen, device="cuda").mul_(std) * tile.repeat_interleave(BLOCK, 1)[:, :c]


def _weights(gen, count, r, c):
    """Codes and factors of `count` matrices in 128 x 128 blocks, one at a time."""
    q = torch.empty(count, r, c, dtype=torch.uint8, device="cuda")
    inv = torch.empty(count, _blocks(r), _blocks(c), device="cuda")
    for i in range(count):
        x = torch.randn(_blocks(r) * BLOCK, _blocks(c) * BLOCK, generator=gen, device="cuda")
        x = x.mul_(0.6 / math.sqrt(c)).view(_blocks(r), BLOCK, _blocks(c), BLOCK)
        x.mul_(torch.randn(_blocks(r), 1, _blocks(c), 1, generator=gen, device="cuda").mul_(0.3).exp_())
        x[-1, r - (_blocks(r) - 1) * BLOCK:] = 0
        x[:, :, -1, c - (_blocks(c) - 1) * BLOCK:] = 0
        scale = 448.0 / x.abs().amax((1, 3), keepdim=True)
        q[i] = (x * scale).to(torch.float8_e4m3fn).view(torch.uint8).view(_blocks(r) * BLOCK, -1)[:r, :c]
        inv[i] = (1.0 / scale)[:, 0, :, 0]
    return q, inv


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda")


def _f32(*shape):
    return torch.zeros(shape, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s, n, nb = {"case": case}, case["n"], _blocks(case["n"])
    if case["op"] == "backward":
        t, tb = case["rows"], _blocks(case["rows"])
        s["dh"] = _rows(gen, t, n, 1e-3).to(OUT[case["grad"]])
        gu = torch.stack([_rows(gen, t, n, 1.0), _rows(gen, t, n, 1.0)], 1)
        q, s["sgu"] = _tiles(gu, *reversed(FP8["e4m3"]))
        s["gu"] = q.view(torch.uint8)
        s["dgu"], s["sdgu"] = _u8(t, 2, n), _f32(t, 2, nb)
        s["dgu_t"], s["sdgu_t"] = _u8(2, n, t), _f32(2, n, tb)
        s["h_t"], s["sh_t"] = _u8(n, t), _f32(n, tb)
        return s
    rows, k = case["m"] if case["op"] == "gated" else case["rows"], case["k"]
    q, s["sx"] = _tiles(_rows(gen, rows, k, 1.0), *reversed(FP8["e4m3"]))
    s["x"] = q.view(torch.uint8)
    experts = 1 if case["op"] == "gated" else case["experts"]
    w, sw = _weights(gen, 2 * experts, n, k)
    shape = (2,) if case["op"] == "gated" else (experts, 2)
    s["w"], s["sw"] = w.view(*shape, n, k), sw.view(*shape, nb, _blocks(k))
    if case["op"] == "experts":
        counts = np.random.RandomState(int(seed) % (1 << 31)).permutation(_counts(case))
        s["ends"] = torch.from_numpy(np.cumsum(counts)).to("cuda")
        s["most"] = int(counts.max())  # the capacity that a padded layout needs
    s["h"], s["sh"] = _u8(rows, n), _f32(rows, nb)
    s["gu"], s["sgu"] = (_u8(rows, 2, n), _f32(rows, 2, nb)) if case["keep"] else (None, None)
    return s


# ------------------------------------------------------------- one pass each

def run(s):
    case = s["case"]
    if own:
        return _own(s)
    return _backward_plain(s) if case["op"] == "backward" else _gated_plain(s)


def _own(s):
    import fp8_scaled_quantization_gb300 as fq
    case = s["case"]
    act = fq.ACT_SILU if case["act"] == "silu" else fq.ACT_GELU_TANH
    e4m3 = FP8["e4m3"][0]
    if case["op"] == "backward":
        fmt, grad = (fq.E4M3, e4m3) if case["fmt"] == "e4m3" else (fq.E5M2, FP8["e5m2"][0])
        fq.fp8_gated_block_backward(s["dh"], s["gu"], s["sgu"], s["dgu"], s["sdgu"], s["dgu_t"], s["sdgu_t"], s["h_t"],
                                    s["sh_t"], fmt_grad=fmt, act=act)
        return {"dgu": s["dgu"].view(grad), "dgu_factors": s["sdgu"], "dgu_t": s["dgu_t"].view(grad),
                "dgu_t_factors": s["sdgu_t"], "h_t": s["h_t"].view(e4m3), "h_t_factors": s["sh_t"]}
    if case["op"] == "gated":
        fq.fp8_gemm_block_gated(s["x"], s["sx"], s["w"], s["sw"], s["h"], s["sh"], s["gu"], s["sgu"], act=act)
    else:
        fq.fp8_gemm_block_gated_grouped(s["x"], s["sx"], s["w"], s["sw"], s["ends"], s["h"], s["sh"], s["gu"], s["sgu"],
                                        act=act)
    out = {"h": s["h"].view(e4m3), "h_factors": s["sh"]}
    if case["keep"]:
        out.update(gu=s["gu"].view(e4m3), gu_factors=s["sgu"])
    return out


def _rows32(q, inv):
    """Dequantized values of 1 x 128 tiles along the last axis."""
    return q.view(FP8["e4m3"][0]).float() * inv.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _blocks32(q, inv):
    r, c = q.shape[-2:]
    f = inv.repeat_interleave(BLOCK, -1)[..., :c].repeat_interleave(BLOCK, -2)[..., :r, :]
    return q.view(FP8["e4m3"][0]).float() * f


def _act32(g, act):
    """The activation and its derivative."""
    if act == "silu":
        y, dy = g, 1.0
    else:
        y, dy = 2 * GELU_C * (g + GELU_CUBE * g * g * g), 2 * GELU_C * (1 + 3 * GELU_CUBE * g * g)
    s = 1 / (1 + torch.exp(-y))
    a = g * s
    return a, s + a * (1 / (1 + torch.exp(y))) * dy


def _gated_plain(s):
    case = s["case"]
    x, w = _rows32(s["x"], s["sx"]), _blocks32(s["w"], s["sw"])
    n = case["n"]
    if case["op"] == "gated":
        gu = (x @ w.view(2 * n, -1).T).view(-1, 2, n)
    else:
        # every expert's rows in a padded block of its own, one batched product, rows taken back
        t, e, most = case["rows"], case["experts"], s["most"]
        row = torch.arange(t, device="cuda")
        group = torch.searchsorted(s["ends"], row, right=True)
        first = torch.cat([s["ends"].new_zeros(1), s["ends"]])[group]
        slot = torch.where(group < e, group * most + row - first, e * most)
        px = torch.zeros(e * most + 1, x.shape[1], device="cuda")
        px[slot] = x
        d = torch.bmm(px[:e * most].view(e, most, -1), w.view(e, 2 * n, -1).transpose(1, 2))
        d = torch.cat([d.view(e * most, -1), d.new_zeros(1, d.shape[2])])
        gu = torch.where((group < e)[:, None], d[slot], 0.0).view(-1, 2, n)
    q, inv = _tiles(_act32(gu[:, 0], case["act"])[0] * gu[:, 1], *reversed(FP8["e4m3"]))
    out = {"h": q, "h_factors": inv}
    if case["keep"]:
        out["gu"], out["gu_factors"] = _tiles(gu, *reversed(FP8["e4m3"]))
    return out


def _backward_plain(s):
    case, dh, gu = s["case"], s["dh"].float(), _rows32(s["gu"], s["sgu"])
    g, u = gu[:, 0], gu[:, 1]
    a, da = _act32(g, case["act"])
    dgu = torch.stack([dh * u * da, dh * a], 1)
    grad, top = FP8[case["fmt"]]
    out = {}
    out["dgu"], out["dgu_factors"] = _tiles(dgu, top, grad)
    out["dgu_t"], out["dgu_t_factors"] = _tiles(dgu.permute(1, 2, 0).contiguous(), top, grad)
    out["h_t"], out["h_t_factors"] = _tiles((a * u).T.contiguous(), *reversed(FP8["e4m3"]))
    return out


# --------------------------------------------------------- the same in 64 bits

def _decoded():
    """The 256 values of E4M3, from its definition: sign, exponent and fraction fields."""
    values = []
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        v = (8 + f) * 2.0 ** (e - 10) if e else f * 2.0 ** -9
        if e == 15 and f == 7:
            v = math.nan
        values.append(-v if code & 128 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _wide(q, inv, block_rows):
    """Dequantized values of a matrix in 64 bits, factors indexed by row and column block."""
    r, c = q.shape
    at = torch.arange(r, device="cuda")[:, None] // block_rows, torch.arange(c, device="cuda")[None, :] // BLOCK
    return _decoded()[q.int()].mul_(inv.double()[at])


def _wide_act(g, act):
    """The activation by the hyperbolic tangent of half its argument, and its derivative."""
    if act == "silu":
        t = torch.tanh(g / 2)
        return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t) * (1 + t) / 4
    z = GELU_C * (g + GELU_CUBE * g ** 3)
    t = torch.tanh(z)
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t) * (1 + t) / 2 * GELU_C * (1 + 3 * GELU_CUBE * g ** 2)


def _wide_tiles(v, top):
    """Values over their tile's factor, not rounded, and the factors amax / top."""
    inv = torch.stack([p.abs().amax(-1) for p in v.split(BLOCK, -1)], -1) / top
    inv[inv == 0] = 1.0
    return v / inv.repeat_interleave(BLOCK, -1)[..., :v.shape[-1]], inv


def exact(case, seed):
    s = prepare(case, seed)
    out = {}
    if case["op"] == "backward":
        if case["rows"] * case["n"] > 1 << 27:  # gigabytes of 64-bit values in each step
            return None
        g, u = _wide(s["gu"][:, 0], s["sgu"][:, 0], 1), _wide(s["gu"][:, 1], s["sgu"][:, 1], 1)
        dh, (a, da) = s["dh"].double(), _wide_act(g, case["act"])
        dg, du, top = dh * u * da, dh * a, FP8[case["fmt"]][1]
        for name, v in (("dgu", (dg, du)), ("dgu_t", (dg.T, du.T))):
            parts = [_wide_tiles(x, top) for x in v]
            axis = 1 if name == "dgu" else 0
            out[name], out[name + "_factors"] = (torch.stack([p[i] for p in parts], axis) for i in (0, 1))
        out["h_t"], out["h_t_factors"] = _wide_tiles((a * u).T, 448.0)
        return out
    rows, n = s["h"].shape
    gu = torch.zeros(rows, 2, n, dtype=torch.float64, device="cuda")
    if case["op"] == "gated":
        spans = [(0, rows, s["w"], s["sw"])]
    else:
        ends = [0] + s["ends"].tolist()
        spans = [(a, b, s["w"][e], s["sw"][e]) for e, (a, b) in enumerate(zip(ends, ends[1:])) if b > a]
    for a, b, w, sw in spans:
        x = _wide(s["x"][a:b], s["sx"][a:b], 1)
        for i in (0, 1):
            gu[a:b, i] = x @ _wide(w[i], sw[i], BLOCK).T
    out["h"], out["h_factors"] = _wide_tiles(_wide_act(gu[:, 0], case["act"])[0] * gu[:, 1], 448.0)
    if case["keep"]:
        out["gu"], out["gu_factors"] = _wide_tiles(gu, 448.0)
    return out


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
