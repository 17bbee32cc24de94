"""GB300-native FP8 scaled quantization.

Python binding of the C ABI in ``include/fp8q.h``.  Every function here only
marshals arguments (tensor data pointers, sizes, the current CUDA stream) and
calls the CUDA library; all arithmetic runs in the library's sm_103a kernels.
Tensors must be contiguous CUDA tensors; BF16 / fp32 inputs, uint8 codes,
fp32 scalars, int64 saturation counters (read as unsigned 64-bit).

Entry points (same names as the C ABI):
  fp8_amax, fp8_update_scale_delayed, fp8_quantize,
  fp8_quantize_cast_transpose, fp8_quantize_block, fp8_dequantize.
"""
from __future__ import annotations

import ctypes
import struct
from operator import attrgetter

import torch

from . import _lib

E4M3, E5M2 = 0, 1
DT_BF16, DT_FP32 = 0, 1
AMAX_MAX, AMAX_MOST_RECENT = 0, 1
COLUMNWISE_FROM_ORIGINAL, COLUMNWISE_FROM_ROWWISE_DEQUANTIZED = 0, 1
B_NK, B_KN = 0, 1
FP8_MAX = {E4M3: 448.0, E5M2: 57344.0}

__all__ = [
    "E4M3", "E5M2", "DT_BF16", "DT_FP32", "AMAX_MAX", "AMAX_MOST_RECENT", "FP8_MAX", "Fp8Error",
    "fp8_amax", "fp8_update_scale_delayed", "fp8_quantize", "fp8_quantize_cast_transpose",
    "fp8_quantize_block", "fp8_dequantize", "fp8_quantize_delayed", "fp8_quantize_mx", "fp8_dequantize_mx",
    "fp8_block128_scales_to_mx", "fp8_amax_noalloc", "fp8_quantize_current", "fp8_quantize_hybrid", "fp8_quantize_block_cast_transpose",
    "fp8_amax_grouped", "fp8_quantize_grouped", "COLUMNWISE_FROM_ORIGINAL", "COLUMNWISE_FROM_ROWWISE_DEQUANTIZED",
    "B_NK", "B_KN", "fp8_gemm_block", "fp8_gemm_block_grouped", "fp8_gemm_block_grouped_wgrad",
    "fp8_grad_norm_grouped", "fp8_grad_clip_grouped",
    "launch_count", "version", "library", "release_stream_workspace", "wait_timeouts",
]


class Fp8Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} [status {status}]")
        self.status = status


def library():
    """The loaded ctypes library (raises if it has not been built)."""
    return _lib.load()


def version() -> int:
    return library().fp8_version()


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(library().fp8_launch_count())


def wait_timeouts() -> int:
    """Waits inside the library's tile pipelines that gave up on the current
    device since the library was loaded (synchronises the device).  Any change
    across a call means that call's outputs are incomplete."""
    import ctypes
    count = ctypes.c_ulonglong(0)
    _check(library().fp8_wait_timeouts(ctypes.addressof(count)))
    return int(count.value)


def release_stream_workspace(stream=None):
    """Free the library's reduction workspace of `stream` (default: the current
    stream) on the current device, after the stream's queued work."""
    _check(library().fp8_release_stream_workspace(_stream(stream)))


def _check(status: int):
    if status != 0:
        msg = library().fp8_last_error_message().decode(errors="replace")
        raise Fp8Error(status, msg)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DT_BF16
    if t.dtype == torch.float32:
        return DT_FP32
    raise TypeError(f"expected a bfloat16 or float32 tensor, got {t.dtype}")


def _p(t) -> int | None:
    """Data pointer of an optional contiguous tensor on the current CUDA device
    (the library launches on the current device's stream, so a tensor on
    another device would be reached through a peer pointer)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"expected a tensor, got {type(t)}")
    if not t.is_cuda:
        raise ValueError("tensors passed to the FP8 library must live on a CUDA device")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensor on {t.device}, but the current CUDA device is cuda:{torch.cuda.current_device()}; "
                         "call inside `with torch.cuda.device(...)`")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the FP8 library must be contiguous")
    return t.data_ptr() or None


def _f32(t, name: str) -> int | None:
    """Pointer of an optional fp32 device scalar (amax, scale, scale_inv): the
    library reads or writes one 4-byte word there."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.numel() < 1:
        raise ValueError(f"{name} must be a float32 tensor of at least one element")
    return _p(t)


def _u64(t, name: str) -> int | None:
    """Pointer of an optional 64-bit device counter (the saturation count)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.int64, torch.uint64) or t.numel() < 1:
        raise ValueError(f"{name} must be an int64 tensor of at least one element")
    return _p(t)


# The current stream's handle without building a Stream object (3 us per call), where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device()) or None
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream or None
    return int(stream) or None


def _rows_cols(x: torch.Tensor):
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"expected a 2-D tensor, got shape {tuple(shape)}")
    return shape[0], shape[1]


def fp8_amax(x, amax_out, fmt=E4M3, margin=0, scale_out=None, scale_inv_out=None, stream=None):
    """amax_out[0] = max|x|; with scale_out / scale_inv_out, also the current scale."""
    _check(library().fp8_amax(_p(x), _dt(x), x.numel(), _f32(amax_out, "amax_out"), fmt, margin,
                              _f32(scale_out, "scale_out"), _f32(scale_inv_out, "scale_inv_out"), _stream(stream)))


def fp8_quantize_mx(x, fmt, q_row=None, scale_row=None, q_col=None, scale_col=None, stream=None):
    """MXFP8: codes with one E8M0 scale per 32 elements, rowwise ([rows, cols] codes,
    [rows, ceil(cols/32)] scales) and/or columnwise (transposed: [cols, rows] codes,
    [cols, ceil(rows/32)] scales)."""
    rows, cols = _rows_cols(x)
    for t, shape in ((q_row, (rows, cols)), (scale_row, (rows, -(-cols // 32))), (q_col, (cols, rows)),
                     (scale_col, (cols, -(-rows // 32)))):
        if t is not None and (t.dtype != torch.uint8 or tuple(t.shape) != shape):
            raise ValueError(f"MX outputs must be uint8 {shape}")
    _check(library().fp8_quantize_mx(_p(x), _dt(x), rows, cols, fmt, _p(q_row), _p(scale_row), _p(q_col),
                                     _p(scale_col), _stream(stream)))


def fp8_dequantize_mx(q, scales, fmt, y, stream=None):
    """y = decode(q) * 2^(scale - 127) for rowwise MX data [rows, cols]."""
    rows, cols = _rows_cols(q)
    if scales.dtype != torch.uint8 or tuple(scales.shape) != (rows, -(-cols // 32)):
        raise ValueError("scales must be uint8 [rows, ceil(cols/32)]")
    if tuple(y.shape) != (rows, cols):
        raise ValueError("y must have q's shape")
    _check(library().fp8_dequantize_mx(_p(q), _p(scales), fmt, rows, cols, _p(y), _dt(y), _stream(stream)))


def fp8_block128_scales_to_mx(scale_inv, rows, cols, mx_scales, bad_blocks_out=None, stream=None):
    """E8M0 1x32 scales from power-of-two 128x128 block scale_inv (codes unchanged)."""
    if scale_inv.dtype != torch.float32 or mx_scales.dtype != torch.uint8:
        raise TypeError("scale_inv must be float32 and mx_scales uint8")
    if tuple(mx_scales.shape) != (rows, -(-cols // 32)):
        raise ValueError("mx_scales must be uint8 [rows, ceil(cols/32)]")
    _check(library().fp8_block128_scales_to_mx(_p(scale_inv), rows, cols, _p(mx_scales),
                                               _u64(bad_blocks_out, "bad_blocks_out"), _stream(stream)))


def fp8_amax_noalloc(x, amax_out, fmt=E4M3, margin=0, scale_out=None, scale_inv_out=None, stream=None):
    """fp8_amax for callers that cannot allocate device memory: the library
    uses a fixed file-scope scratch array instead of a per-stream workspace.
    At most 2**28 elements; make the first call on a device before any stream
    capture; calls that overlap on the GPU race on the shared scratch."""
    _check(library().fp8_amax_noalloc(_p(x), _dt(x), x.numel(), _f32(amax_out, "amax_out"), fmt, margin,
                                      _f32(scale_out, "scale_out"), _f32(scale_inv_out, "scale_inv_out"),
                                      _stream(stream)))


def fp8_update_scale_delayed(amax_history, step, new_amax, algo, fmt, margin, scale_out, scale_inv_out,
                             stream=None):
    """Delayed-scaling update of a float32 history (in place) -> scale_out, scale_inv_out."""
    if amax_history.dtype != torch.float32:
        raise TypeError("amax_history must be float32")
    _check(library().fp8_update_scale_delayed(_p(amax_history), amax_history.numel(), int(step),
                                              _f32(new_amax, "new_amax"), algo, fmt, margin,
                                              _f32(scale_out, "scale_out"), _f32(scale_inv_out, "scale_inv_out"),
                                              _stream(stream)))


def fp8_quantize(x, fmt, scale, q_out, amax_out=None, sat_count_out=None, stream=None):
    """q_out = FP8 codes of x * scale; optional fused amax and saturation count."""
    if q_out.dtype != torch.uint8:
        raise TypeError("q_out must be uint8")
    if q_out.numel() != x.numel():
        raise ValueError("q_out must have as many elements as x")
    _check(library().fp8_quantize(_p(x), _dt(x), x.numel(), fmt, _f32(scale, "scale"), _p(q_out),
                                  _f32(amax_out, "amax_out"), _u64(sat_count_out, "sat_count_out"),
                                  _stream(stream)))


def fp8_quantize_delayed(x, fmt, scale, scale_inv, q_out, amax_history, step, algo=AMAX_MAX, margin=0,
                         amax_out=None, sat_count_out=None, stream=None):
    """One delayed-scaling step in one call (the cast, then a one-CTA finalize):
    q_out = codes of x * scale, then
    amax(x) goes into amax_history[step % len] and scale / scale_inv are
    overwritten with the scale of the next step."""
    if q_out.dtype != torch.uint8 or q_out.numel() != x.numel():
        raise ValueError("q_out must be uint8 with as many elements as x")
    if amax_history.dtype != torch.float32:
        raise TypeError("amax_history must be float32")
    _check(library().fp8_quantize_delayed(_p(x), _dt(x), x.numel(), fmt, _f32(scale, "scale"),
                                          _f32(scale_inv, "scale_inv"), _p(q_out), _p(amax_history),
                                          amax_history.numel(), int(step), algo, margin, _f32(amax_out, "amax_out"),
                                          _u64(sat_count_out, "sat_count_out"), _stream(stream)))


def fp8_quantize_cast_transpose(x, fmt, scale, q_row, q_col, amax_out=None, stream=None):
    """Rowwise [rows, cols] and columnwise [cols, rows] codes under one scale."""
    rows, cols = _rows_cols(x)
    if q_row is not None and (q_row.dtype != torch.uint8 or tuple(q_row.shape) != (rows, cols)):
        raise ValueError("q_row must be uint8 [rows, cols]")
    if q_col is not None and (q_col.dtype != torch.uint8 or tuple(q_col.shape) != (cols, rows)):
        raise ValueError("q_col must be uint8 [cols, rows]")
    _check(library().fp8_quantize_cast_transpose(_p(x), _dt(x), rows, cols, fmt, _f32(scale, "scale"), _p(q_row),
                                                 _p(q_col), _f32(amax_out, "amax_out"), _stream(stream)))


def fp8_quantize_block(x, block_rows, block_cols, fmt, q_out, scale_inv_out, stream=None):
    """Block-scaled codes and per-block scale_inv ([ceil(r/br), ceil(c/bc)] fp32)."""
    rows, cols = _rows_cols(x)
    if q_out.dtype != torch.uint8 or tuple(q_out.shape) != (rows, cols):
        raise ValueError("q_out must be uint8 [rows, cols]")
    if block_rows > 0 and block_cols > 0:
        want = (-(-rows // block_rows), -(-cols // block_cols))
        if scale_inv_out.dtype != torch.float32 or tuple(scale_inv_out.shape) != want:
            raise ValueError(f"scale_inv_out must be float32 {want}")
    _check(library().fp8_quantize_block(_p(x), _dt(x), rows, cols, block_rows, block_cols, fmt, _p(q_out),
                                        _p(scale_inv_out), _stream(stream)))


def fp8_dequantize(q, fmt, scale_inv, y, block_rows=0, block_cols=0, stream=None):
    """y = decode(q) * scale_inv (fp32 multiply) stored as y's dtype (bf16 / fp32)."""
    if q.dtype != torch.uint8:
        raise TypeError("q must be uint8")
    if y.numel() != q.numel():
        raise ValueError("y must have as many elements as q")
    if q.dim() == 2:
        rows, cols = int(q.shape[0]), int(q.shape[1])
    else:
        if block_rows or block_cols:
            raise ValueError("block-scaled dequantize needs a 2-D q")
        rows, cols = 1, q.numel()
    if block_rows > 0 and block_cols > 0:
        nblocks = -(-rows // block_rows) * -(-cols // block_cols)
        if scale_inv.dtype != torch.float32 or scale_inv.numel() < nblocks:
            raise ValueError(f"block scale_inv must be float32 with at least {nblocks} elements")
        si = _p(scale_inv)
    else:
        si = _f32(scale_inv, "scale_inv")
    _check(library().fp8_dequantize(_p(q), fmt, rows, cols, si, block_rows, block_cols, _p(y),
                                    _dt(y), _stream(stream)))


def fp8_quantize_hybrid(x, fmt_row, scale_row, q_row, fmt_col, scale_col, q_col,
                        source=COLUMNWISE_FROM_ORIGINAL, stream=None):
    """Rowwise codes (fmt_row, scale_row) and transposed columnwise codes (fmt_col,
    scale_col) from x or from the BF16-dequantized rowwise value."""
    rows, cols = _rows_cols(x)
    if q_row.dtype != torch.uint8 or tuple(q_row.shape) != (rows, cols):
        raise ValueError("q_row must be uint8 [rows, cols]")
    if q_col.dtype != torch.uint8 or tuple(q_col.shape) != (cols, rows):
        raise ValueError("q_col must be uint8 [cols, rows]")
    _check(library().fp8_quantize_hybrid(_p(x), _dt(x), rows, cols, fmt_row, _f32(scale_row, "scale_row"),
                                         _p(q_row), fmt_col, _f32(scale_col, "scale_col"), _p(q_col), source,
                                         _stream(stream)))


def fp8_quantize_block_cast_transpose(x, fmt, q_row=None, scale_inv_row=None, q_col=None, scale_inv_col=None,
                                      stream=None):
    """1 x 128 blockwise codes of x ([rows, cols] + fp32 [rows, ceil(cols/128)]) and of
    x^T ([cols, rows] + fp32 [cols, ceil(rows/128)]) from one read of x."""
    rows, cols = _rows_cols(x)
    for t, shape, dt in ((q_row, (rows, cols), torch.uint8), (scale_inv_row, (rows, -(-cols // 128)), torch.float32),
                         (q_col, (cols, rows), torch.uint8), (scale_inv_col, (cols, -(-rows // 128)), torch.float32)):
        if t is not None and (t.dtype != dt or tuple(t.shape) != shape):
            raise ValueError(f"block cast-transpose outputs must be {dt} {shape}")
    _check(library().fp8_quantize_block_cast_transpose(_p(x), _dt(x), rows, cols, fmt, _p(q_row), _p(scale_inv_row),
                                                       _p(q_col), _p(scale_inv_col), _stream(stream)))


def _ptr_array(tensors):
    return (ctypes.c_void_p * len(tensors))(*[_p(t) for t in tensors])


def fp8_amax_grouped(xs, amax_out=None, fmt=E4M3, margin=0, scale_out=None, scale_inv_out=None, stream=None):
    """Per-tensor amax (and current scale) of up to 128 tensors in one launch (+ finalize);
    outputs are float32 device tensors of at least len(xs) elements."""
    if not xs or len({t.dtype for t in xs}) != 1:
        raise ValueError("xs must be a non-empty list of tensors of one dtype")
    for out in (amax_out, scale_out, scale_inv_out):
        if out is not None and (out.dtype != torch.float32 or out.numel() < len(xs)):
            raise ValueError("grouped outputs must be float32 tensors of at least len(xs) elements")
    ns = (ctypes.c_int64 * len(xs))(*[t.numel() for t in xs])
    _check(library().fp8_amax_grouped(len(xs), _ptr_array(xs), ns, _dt(xs[0]), _p(amax_out), fmt, margin,
                                      _p(scale_out), _p(scale_inv_out), _stream(stream)))


def fp8_quantize_grouped(xs, fmt, scales, qs, stream=None):
    """qs[i] = codes of xs[i] * scales[i] for up to 128 tensors in one kernel launch."""
    if not xs or len(xs) != len(qs) or len({t.dtype for t in xs}) != 1:
        raise ValueError("xs and qs must be equally long lists; xs of one dtype")
    for x, q in zip(xs, qs):
        if q.dtype != torch.uint8 or q.numel() != x.numel():
            raise ValueError("each q must be uint8 with as many elements as its x")
    if scales.dtype != torch.float32 or scales.numel() < len(xs):
        raise ValueError("scales must be a float32 tensor of at least len(xs) elements")
    ns = (ctypes.c_int64 * len(xs))(*[t.numel() for t in xs])
    _check(library().fp8_quantize_grouped(len(xs), _ptr_array(xs), ns, _dt(xs[0]), fmt, _p(scales), _ptr_array(qs),
                                          _stream(stream)))


def fp8_quantize_current(x, fmt, q_out, margin=0, amax_out=None, scale_out=None, scale_inv_out=None, stream=None):
    """Current scaling in one call: amax(x), the scale with `margin`, and q_out = codes
    of x * scale (the cast reduces the amax partials itself; no separate finalize)."""
    if q_out.dtype != torch.uint8:
        raise TypeError("q_out must be uint8")
    if q_out.numel() != x.numel():
        raise ValueError("q_out must have as many elements as x")
    _check(library().fp8_quantize_current(_p(x), _dt(x), x.numel(), fmt, margin, _p(q_out),
                                          _f32(amax_out, "amax_out"), _f32(scale_out, "scale_out"),
                                          _f32(scale_inv_out, "scale_inv_out"), _stream(stream)))


def _operand(q, scale_inv, shape, scale_shape, name):
    """Shape and type checks of one operand of a product."""
    if q.dtype is not torch.uint8 or q.shape != shape:
        raise ValueError(f"{name} must be uint8 {shape}")
    if scale_inv.dtype is not torch.float32 or scale_inv.shape != scale_shape:
        raise ValueError(f"scale_inv_{name} must be float32 {scale_shape}")


def _ptrs(*tensors):
    """Data pointers of contiguous tensors on the current CUDA device (one look at the device for all)."""
    here = torch.cuda.current_device() if tensors[0].is_cuda else None
    out = []
    for t in tensors:
        if t.get_device() != here or not t.is_contiguous():
            _p(t)  # says what is wrong with it
        out.append(t.data_ptr() or None)
    return out


def _ends(group_ends):
    if group_ends.dtype != torch.int64 or group_ends.dim() != 1:
        raise ValueError("group_ends must be a 1-D int64 tensor")
    return group_ends.shape[0]


def _out(d, rows):
    """Columns of an output [rows, n]."""
    shape = d.shape
    if len(shape) != 2 or shape[0] != rows:
        raise ValueError(f"d must be [{rows}, n]")
    return shape[1]


def fp8_gemm_block(a, scale_inv_a, b, scale_inv_b, d, fmt_a=E4M3, fmt_b=E4M3, b_layout=B_NK, b_block_rows=128,
                   accumulate=False, stream=None):
    """d[m, n] = the product of block-scaled operands: a [m, k] codes with 1 x 128 factors,
    b [n, k] (B_NK) or [k, n] (B_KN) codes with 128 x 128 factors (or, with b_block_rows=1
    and B_NK, 1 x 128 factors).  d is bfloat16 or float32; accumulate adds to a float32 d."""
    m, k = _rows_cols(a)
    n = _out(d, m)
    kb = -(-k // 128)
    rows_b = n if b_block_rows == 1 else -(-n // 128)
    _operand(a, scale_inv_a, (m, k), (m, kb), "a")
    if b_layout == B_KN:
        _operand(b, scale_inv_b, (k, n), (kb, rows_b), "b")
    else:
        _operand(b, scale_inv_b, (n, k), (rows_b, kb), "b")
    pa, psa, pb, psb, pd = _ptrs(a, scale_inv_a, b, scale_inv_b, d)
    _check(library().fp8_gemm_block(pa, fmt_a, psa, pb, fmt_b, psb, b_layout, b_block_rows, m, n, k, pd, _dt(d),
                                    1 if accumulate else 0, _stream(stream)))


def fp8_gemm_block_grouped(a, scale_inv_a, b, scale_inv_b, group_ends, d, fmt_a=E4M3, fmt_b=E4M3, b_layout=B_NK,
                           stream=None):
    """The product per expert over rows sorted by expert: rows group_ends[e-1] .. group_ends[e]-1
    of a [rows, k] times b[e] ([groups, n, k], or [groups, k, n] with B_KN) into d [rows, n];
    rows after the last end become zeros.  group_ends: int64 on the device."""
    rows, k = _rows_cols(a)
    groups = _ends(group_ends)
    n = _out(d, rows)
    kb, nb = -(-k // 128), -(-n // 128)
    shape, scales = ((groups, k, n), (groups, kb, nb)) if b_layout == B_KN else ((groups, n, k), (groups, nb, kb))
    _operand(a, scale_inv_a, (rows, k), (rows, kb), "a")
    _operand(b, scale_inv_b, shape, scales, "b")
    ends, pa, psa, pb, psb, pd = _ptrs(group_ends, a, scale_inv_a, b, scale_inv_b, d)
    _check(library().fp8_gemm_block_grouped(groups, ends, pa, fmt_a, psa, pb, fmt_b, psb, b_layout, rows, n, k, pd,
                                            _dt(d), _stream(stream)))


def fp8_gemm_block_grouped_wgrad(a, scale_inv_a, b, scale_inv_b, group_ends, d, fmt_a=E4M3, fmt_b=E4M3,
                                 accumulate=False, stream=None):
    """One weight gradient per expert: d[e] [m, n] = sum over the rows of expert e of
    a [m, rows] times b [n, rows], both with 1 x 128 factors along the rows."""
    m, rows = _rows_cols(a)
    n, _ = _rows_cols(b)
    groups = _ends(group_ends)
    if d.shape != (groups, m, n):
        raise ValueError(f"d must be [{groups}, {m}, {n}]")
    rb = -(-rows // 128)
    _operand(a, scale_inv_a, (m, rows), (m, rb), "a")
    _operand(b, scale_inv_b, (n, rows), (n, rb), "b")
    ends, pa, psa, pb, psb, pd = _ptrs(group_ends, a, scale_inv_a, b, scale_inv_b, d)
    _check(library().fp8_gemm_block_grouped_wgrad(groups, ends, pa, fmt_a, psa, pb, fmt_b, psb, m, n, rows, pd, _dt(d),
                                                  int(accumulate), _stream(stream)))


_GRAD_DTYPES = {torch.bfloat16: DT_BF16, torch.float32: DT_FP32}


_dtype_of = attrgetter("dtype")


def _pack(code, values):
    """Host array of a C type as bytes (a pointer argument takes them as they are)."""
    return struct.pack(f"{len(values)}{code}", *values)


def _grad_table(tensors, name):
    """Host arrays (pointers, dtypes) of a list of contiguous BF16 / fp32 tensors on the current device."""
    here = torch.cuda.current_device() if tensors[0].is_cuda else None
    if set(map(torch.Tensor.get_device, tensors)) != {here} or not all(map(torch.Tensor.is_contiguous, tensors)):
        for t in tensors:
            _p(t)  # says what is wrong with the first one
    kinds = list(map(_dtype_of, tensors))
    if not set(kinds) <= _GRAD_DTYPES.keys():
        raise TypeError(f"{name} must be bfloat16 or float32 tensors")
    dtypes = [_GRAD_DTYPES[kinds[0]]] * len(kinds) if len(set(kinds)) == 1 else [_GRAD_DTYPES[k] for k in kinds]
    return _pack("Q", list(map(torch.Tensor.data_ptr, tensors))), _pack("i", dtypes)


def fp8_grad_norm_grouped(xs, norm_out, stream=None):
    """norm_out[0] = sqrt of the sum of squares over all elements of all tensors in xs."""
    if not xs:
        raise ValueError("xs must be a non-empty list of tensors")
    ptrs, dtypes = _grad_table(xs, "xs")
    ns = list(map(torch.Tensor.numel, xs))
    _check(library().fp8_grad_norm_grouped(len(xs), ptrs, _pack("q", ns), dtypes, _f32(norm_out, "norm_out"),
                                           _stream(stream)))


def fp8_grad_clip_grouped(xs, max_norm, norm_out=None, ys=None, coef_out=None, eps=1e-6, stream=None):
    """ys[i] = xs[i] * min(1, max_norm / (norm + eps)), norm over all tensors of xs; in place
    without ys.  A norm that is NaN or Inf leaves the values as they are."""
    if not xs or (ys is not None and len(ys) != len(xs)):
        raise ValueError("xs must be a non-empty list of tensors, and ys as long as xs")
    ns = list(map(torch.Tensor.numel, xs))
    if ys is not None and list(map(torch.Tensor.numel, ys)) != ns:
        raise ValueError("each y must have as many elements as its x")
    ptrs, dtypes = _grad_table(xs, "xs")
    outs, out_dtypes = _grad_table(ys, "ys") if ys is not None else (None, None)
    _check(library().fp8_grad_clip_grouped(len(xs), ptrs, _pack("q", ns), dtypes, outs, out_dtypes, max_norm, eps,
                                           _f32(norm_out, "norm_out"), _f32(coef_out, "coef_out"), _stream(stream)))
