"""Python binding of libfp8blk: FP8 (E4M3) blockwise quantisation and GEMM on B200.

Argument marshalling only.  Every step runs in the library's CUDA kernels;
torch provides device memory and the current stream.  There is no CPU
fallback: importing this package without the built library (and without
nvcc to build it) raises, and every call on a non-CUDA tensor raises.

The functions carry the C-ABI's names (include/fp8blk.h).  Output tensors
may be passed in (they must be contiguous CUDA tensors of the right dtype
and shape); missing ones are allocated with torch.empty, on the stream of
the call: the current one, or the one passed as ``stream`` (a
torch.cuda.Stream or a cudaStream_t handle).  A stream that is passed in is
ordered against no other stream by the call: the caller orders the inputs
before it and keeps them until it is done.

Layouts (row-major, dimensions multiples of 128):
  fp8blk_quantize_act_1x128(x[R,C], mode)
      ROWWISE   -> q_row[R,C] float8_e4m3fn, s_row[C/128,R] float32
      COLWISE_T -> q_colT[C,R],              s_colT[R/128,C]
      BOTH      -> all four
  fp8blk_quantize_weight_128x128(w[N,K])   -> q[N,K],  s[N/128,K/128]
  fp8blk_quantize_weight_128x128_t(w[N,K]) -> qT[K,N], sT[K/128,N/128]
  fp8blk_quantize_weight_128x128_both(w[N,K]) -> q, s, qT, sT from one read of w
  fp8blk_gemm(layout, a[M,K], sa[K/128,M], b[N,K], sb) -> d[M,N] bfloat16
      sb = [N/128,K/128] for FWD/DGRAD, [K/128,N] for WGRAD

Rows sorted by group (tokens sorted by expert; offsets: int32 [groups + 1] on the device, any
number of rows in a group):
  fp8blk_quantize_act_1x128_grouped(x[T,C], offsets, mode)
      ROWWISE   -> q_row[T,C], s_row[C/128,T];  COLWISE_T -> q_colT[C,P], s_colT[P/128,C],
      P = fp8blk_grouped_padded_rows(T, groups): whole 128-token blocks for every group
  fp8blk_gemm_grouped(layout, a, sa, b, sb, offsets)
      FWD  : a[T,in],  b = q[groups*out,in]            -> Y[T,out]
      DGRAD: a[T,out], b = qT[in,groups*out]           -> dX[T,in]
      WGRAD: a[out,P], b[in,P]                         -> dW[groups,out,in]
  fp8blk_linear_grouped(x[T,in], q, s, offsets) -> Y[T,out], x quantised on the way

4-bit microscaled formats (MXFP4, NVFP4; codes and scales as uint8, two codes to a byte):
  fp8blk_quantize_mx4(x[R,C], fmt, mode)
      ROWWISE   -> q_row[R,C/2],  s_row[ceil(R/128), ceil(C/(4 block)), 512]
      COLWISE_T -> q_colT[C,P/2], s_colT for [C,P], P = R rounded up to a multiple of 32
  fp8blk_dequantize_mx4(q, s, fmt) -> bf16 values
  fp8blk_gemm_mx4(a[M,K/2], sa, b[N,K/2], sb, fmt) -> d[M,N]
  fp8blk_linear_mx4(x[M,K], qw[N,K/2], sw, fmt)    -> d[M,N], x quantised on the way
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import (A_E5M2, B_E5M2, BOTH, COLWISE_T, DGRAD, E5M2, FWD, MAX_GROUPS, MAX_WEIGHTS, MXFP4, NVFP4, OUT_F32, ROWWISE,
                   WGRAD,
                   Fp8BlkError, LIB_PATH, WeightDesc, check, lib, status_string)

__all__ = [
    "fp8blk_quantize_act_1x128", "fp8blk_quantize_weight_128x128", "fp8blk_quantize_weight_128x128_t",
    "fp8blk_quantize_weight_128x128_both", "fp8blk_quantize_weights_128x128_both", "fp8blk_amax_ema", "fp8blk_amax_ema_workspace_bytes",
    "fp8blk_amax_ema_static", "AMAX_EMA_STATIC_MAX_ROWS",
    "fp8blk_quantize_tensor", "fp8blk_gemm_tensor_scaled", "fp8_linear_delayed_forward",
    "fp8blk_gemm", "fp8blk_gemm_splitk", "fp8blk_gemm_splitk_count", "fp8blk_gemm_splitk_workspace_bytes", "fp8blk_round_f32_to_bf16", "fp8blk_get_device_error", "fp8blk_version", "linear_forward",
    "linear_backward", "fp8blk_grouped_padded_rows", "fp8blk_quantize_act_1x128_grouped", "fp8blk_gemm_grouped",
    "fp8blk_linear_grouped", "fp8blk_linear_grouped_workspace_bytes",
    "grouped_linear_forward", "grouped_linear_backward", "MAX_GROUPS", "fp8blk_mx4_scale_bytes", "fp8blk_quantize_mx4",
    "fp8blk_dequantize_mx4", "fp8blk_gemm_mx4", "fp8blk_linear_mx4", "fp8blk_linear_mx4_workspace_bytes", "mx4_linear_forward", "mx4_linear_wgrad", "mx4_linear_backward",
    "MXFP4", "NVFP4", "ROWWISE", "COLWISE_T", "BOTH", "E5M2", "FWD", "DGRAD", "WGRAD", "A_E5M2", "B_E5M2",
    "OUT_F32", "MAX_WEIGHTS", "Fp8BlkError",
    "LIB_PATH", "status_string",
]

E4M3 = torch.float8_e4m3fn
E5M2_DTYPE = torch.float8_e5m2


def _stream_handle(stream, device=None) -> int:
    """The cudaStream_t to launch on: `stream`, else the current stream of `device`."""
    if stream is None:
        # The current stream's handle, without a Stream object: every call of the library asks for it.
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device.index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _need_cuda(*tensors) -> torch.device:
    """All given tensors must be CUDA tensors of one device; returns it."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("fp8blk runs on CUDA tensors only (no CPU fallback)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    return dev


def _run(device, fn, *args) -> None:
    """Calls a C entry point with `device` current, so that the library's device
    check, its per-device state and the launch all refer to the tensors' GPU."""
    if device.index == torch._C._cuda_getDevice():
        check(fn(*args))
    else:
        with torch.cuda.device(device):
            check(fn(*args))


def _empty(shape, dtype, device):
    """torch.empty for a contiguous tensor, by the entry point that costs the host least."""
    if len(shape) == 2:
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)
    if len(shape) == 1:
        return torch.empty_strided(shape, (1,), dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _out(t, shape, dtype, device):
    if t is None:
        return _empty(shape, dtype, device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"output must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _pitch(t, width: int) -> int:
    """Row pitch of a 2-D (or the last two dimensions of a) tensor; a single row's stride says nothing, so that
    its pitch is the next one the library takes."""
    return t.stride(-2) if t.shape[-2] > 1 else -(-width // 8) * 8


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _bf16_2d(x):
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("input must be a 2-D bfloat16 tensor with unit column stride")
    return x


def _record(out, stream) -> None:
    """Marks a result (a tensor, None, or a tuple or list of results) as used by `stream`."""
    if isinstance(out, (tuple, list)):
        for t in out:
            _record(t, stream)
    elif out is not None:
        out.record_stream(stream)


def _on_stream(stream, device, call):
    """call() with `stream` current: what it allocates is that stream's memory, which no earlier work of
    another stream still uses, and its results' memory is not given out again before the work that the
    caller's current stream has for them is done."""
    if not isinstance(stream, torch.cuda.Stream):
        # Handles 0 and 1 are the legacy default stream (NULL and cudaStreamLegacy).  ExternalStream would take 0 for
        # "no handle given" and make a stream of its own, and 1 for an identifier of its own streams.
        handle = int(stream)
        stream = torch.cuda.default_stream(device) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device=device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        out = call()
    _record(out, caller)
    return out


def _some_missing(mode, q_row, s_row, q_colT, s_colT) -> bool:
    """Whether a quantiser of that mode has to make an output."""
    return bool(mode & ROWWISE and (q_row is None or s_row is None) or
                mode & COLWISE_T and (q_colT is None or s_colT is None))


def _same_tokens(x, dy) -> None:
    """Padded along the tokens, operands of different numbers of them can look alike."""
    if x.shape[0] != dy.shape[0]:
        raise ValueError("X and dY disagree on their tokens")


def fp8blk_quantize_act_1x128(x, mode=ROWWISE, q_row=None, s_row=None, q_colT=None, s_colT=None,
                              stream=None):
    """Activation quantisation in 1x128 groups.  Returns (q_row, s_row, q_colT, s_colT); unused are None.
    ``mode`` may include E5M2 (codes as torch.float8_e5m2, for gradients)."""
    x = _bf16_2d(x)
    dev = _need_cuda(x)
    if stream is not None and _some_missing(mode, q_row, s_row, q_colT, s_colT):
        return _on_stream(stream, dev, lambda: fp8blk_quantize_act_1x128(x, mode, q_row, s_row, q_colT, s_colT))
    rows, cols = x.shape
    code_dtype = E5M2_DTYPE if mode & E5M2 else E4M3
    if mode & ROWWISE:
        q_row = _out(q_row, (rows, cols), code_dtype, dev)
        s_row = _out(s_row, (cols // 128, rows), torch.float32, dev)
    else:
        q_row = s_row = None
    if mode & COLWISE_T:
        q_colT = _out(q_colT, (cols, rows), code_dtype, dev)
        s_colT = _out(s_colT, (rows // 128, cols), torch.float32, dev)
    else:
        q_colT = s_colT = None
    _run(dev, lib.fp8blk_quantize_act_1x128, _ptr(x), rows, cols, x.stride(0), int(mode), _ptr(q_row), _ptr(s_row),
                                        _ptr(q_colT), _ptr(s_colT), _stream_handle(stream, dev))
    return q_row, s_row, q_colT, s_colT


def fp8blk_quantize_weight_128x128(w, q=None, s=None, stream=None):
    """Weight quantisation in 128x128 blocks.  Returns (q[N,K], s[N/128,K/128])."""
    w = _bf16_2d(w)
    dev = _need_cuda(w)
    if stream is not None and any(t is None for t in (q, s)):
        return _on_stream(stream, dev, lambda: fp8blk_quantize_weight_128x128(w, q, s))
    n, k = w.shape
    q = _out(q, (n, k), E4M3, w.device)
    s = _out(s, (n // 128, k // 128), torch.float32, w.device)
    _run(dev, lib.fp8blk_quantize_weight_128x128, _ptr(w), n, k, w.stride(0), _ptr(q), _ptr(s), _stream_handle(stream, dev))
    return q, s


def fp8blk_quantize_weight_128x128_t(w, qT=None, sT=None, stream=None):
    """The same blocks written transposed.  Returns (qT[K,N], sT[K/128,N/128])."""
    w = _bf16_2d(w)
    dev = _need_cuda(w)
    if stream is not None and any(t is None for t in (qT, sT)):
        return _on_stream(stream, dev, lambda: fp8blk_quantize_weight_128x128_t(w, qT, sT))
    n, k = w.shape
    qT = _out(qT, (k, n), E4M3, w.device)
    sT = _out(sT, (k // 128, n // 128), torch.float32, w.device)
    _run(dev, lib.fp8blk_quantize_weight_128x128_t, _ptr(w), n, k, w.stride(0), _ptr(qT), _ptr(sT),
                                               _stream_handle(stream, dev))
    return qT, sT


def fp8blk_quantize_weight_128x128_both(w, q=None, s=None, qT=None, sT=None, stream=None):
    """Both block layouts from one read of w.  Returns (q[N,K], s[N/128,K/128], qT[K,N], sT[K/128,N/128])."""
    w = _bf16_2d(w)
    dev = _need_cuda(w)
    if stream is not None and any(t is None for t in (q, s, qT, sT)):
        return _on_stream(stream, dev, lambda: fp8blk_quantize_weight_128x128_both(w, q, s, qT, sT))
    n, k = w.shape
    q = _out(q, (n, k), E4M3, w.device)
    s = _out(s, (n // 128, k // 128), torch.float32, w.device)
    qT = _out(qT, (k, n), E4M3, w.device)
    sT = _out(sT, (k // 128, n // 128), torch.float32, w.device)
    _run(dev, lib.fp8blk_quantize_weight_128x128_both, _ptr(w), n, k, w.stride(0), _ptr(q), _ptr(s), _ptr(qT), _ptr(sT),
                                                  _stream_handle(stream, dev))
    return q, s, qT, sT


def fp8blk_gemm_splitk_count(layout, m: int, n: int, k: int) -> int:
    """The split-K count the library picks for this GEMM shape on the current device (1 = none)."""
    return int(lib.fp8blk_gemm_splitk_count(int(layout), int(m), int(n), int(k)))


def fp8blk_gemm_splitk_workspace_bytes(layout, m: int, n: int, k: int, splits: int) -> int:
    """Bytes of workspace fp8blk_gemm_splitk needs for this shape and split count on the current device."""
    return int(lib.fp8blk_gemm_splitk_workspace_bytes(int(layout), int(m), int(n), int(k), int(splits)))


def fp8blk_gemm(layout, a, sa, b, sb, d=None, stream=None, out_dtype=torch.bfloat16, splits=1, workspace=None):
    """Blockwise-scaled E4M3 GEMM, D[M,N] = dequant(A) . dequant(B)^T in bf16 (or, with
    out_dtype=torch.float32 or an fp32 d, the unrounded fp32 sums).  splits > 1 (or "auto":
    fp8blk_gemm_splitk_count) divides each output tile's K range among that many units whose
    fp32 partials are summed in split order; workspace: a float32 CUDA tensor of at least
    fp8blk_gemm_splitk_workspace_bytes(...) bytes (allocated here when None)."""
    dev = _need_cuda(a, sa, b, sb, d)
    if stream is not None and (d is None or (workspace is None and splits != 1)):
        return _on_stream(stream, dev, lambda: fp8blk_gemm(layout, a, sa, b, sb, d, None, out_dtype, splits, workspace))
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k:
        raise ValueError("A and B disagree on K")
    if a.dtype not in (E4M3, E5M2_DTYPE) or b.dtype not in (E4M3, E5M2_DTYPE):
        raise ValueError("A and B must be float8_e4m3fn or float8_e5m2")
    want_sb = (k // 128, n) if layout == WGRAD else (n // 128, k // 128)
    if tuple(sa.shape) != (k // 128, m) or tuple(sb.shape) != want_sb:
        raise ValueError(f"scale shapes {tuple(sa.shape)}, {tuple(sb.shape)} do not match layout {layout}")
    if sa.dtype != torch.float32 or sb.dtype != torch.float32:
        raise ValueError("scales must be float32")
    if not (a.is_contiguous() and b.is_contiguous() and sa.is_contiguous() and sb.is_contiguous()):
        raise ValueError("operands and scales must be contiguous")
    if d is None:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        d = torch.empty((m, n), dtype=out_dtype, device=a.device)
    elif d.dtype not in (torch.bfloat16, torch.float32) or d.dim() != 2 or d.stride(1) != 1 or tuple(d.shape) != (m, n):
        raise ValueError("d must be a bfloat16 or float32 [M,N] tensor with unit column stride")
    flags = (A_E5M2 if a.dtype == E5M2_DTYPE else 0) | (B_E5M2 if b.dtype == E5M2_DTYPE else 0)
    flags |= OUT_F32 if d.dtype == torch.float32 else 0
    if splits == "auto":
        with torch.cuda.device(dev):
            splits = fp8blk_gemm_splitk_count(layout, m, n, k)
    splits = int(splits)
    if splits == 1:
        _run(dev, lib.fp8blk_gemm, int(layout) | flags, m, n, k, _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d),
             d.stride(0), _stream_handle(stream, dev))
        return d
    if workspace is None:
        with torch.cuda.device(dev):
            need = fp8blk_gemm_splitk_workspace_bytes(layout, m, n, k, splits)
        if need < 0:
            raise ValueError("invalid split-K arguments for this device")
        workspace = torch.empty(max(need // 4, 4), dtype=torch.float32, device=a.device)
    elif workspace.dtype != torch.float32 or not workspace.is_contiguous() or workspace.device != a.device:
        raise ValueError("workspace must be a contiguous float32 tensor on the operands' device")
    _run(dev, lib.fp8blk_gemm_splitk, int(layout) | flags, m, n, k, _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d),
         d.stride(0), splits, _ptr(workspace), workspace.numel() * 4, _stream_handle(stream, dev))
    return d


def fp8blk_gemm_splitk(layout, a, sa, b, sb, splits, d=None, workspace=None, stream=None, out_dtype=torch.bfloat16):
    """fp8blk_gemm with split-K over `splits` units per output tile (an int, or "auto")."""
    return fp8blk_gemm(layout, a, sa, b, sb, d=d, stream=stream, out_dtype=out_dtype, splits=splits,
                       workspace=workspace)


def fp8blk_round_f32_to_bf16(x, y=None, stream=None):
    """y = bf16(x) (round to nearest even), elementwise; x a contiguous float32 CUDA tensor."""
    dev = _need_cuda(x, y)
    if stream is not None and y is None:
        return _on_stream(stream, dev, lambda: fp8blk_round_f32_to_bf16(x))
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 tensor")
    y = _out(y, tuple(x.shape), torch.bfloat16, x.device)
    _run(dev, lib.fp8blk_round_f32_to_bf16, _ptr(x), x.numel(), _ptr(y), _stream_handle(stream, dev))
    return y


def fp8blk_quantize_weights_128x128_both(weights, outs=None, stream=None):
    """Both 128x128 block layouts of several weights in one launch.  weights: a list of
    [N,K] bf16 CUDA tensors (row stride may exceed K); outs: None or a list of (q, s, qT, sT)
    per weight.  Returns the list of (q, s, qT, sT), bitwise those of
    fp8blk_quantize_weight_128x128_both on each weight."""
    weights = list(weights)
    if not 1 <= len(weights) <= MAX_WEIGHTS:
        raise ValueError(f"between 1 and {MAX_WEIGHTS} weights per launch")
    outs = list(outs) if outs is not None else [None] * len(weights)
    if len(outs) != len(weights):
        raise ValueError("one output tuple per weight")
    weights = [_bf16_2d(w) for w in weights]
    flat = [t for w, o in zip(weights, outs) for t in (w, *(o or ()))]
    dev = _need_cuda(*flat)
    if stream is not None and any(o is None or any(t is None for t in o) for o in outs):
        return _on_stream(stream, dev, lambda: fp8blk_quantize_weights_128x128_both(weights, outs))
    descs = (WeightDesc * len(weights))()
    result = []
    for i, (w, o) in enumerate(zip(weights, outs)):
        n, k = w.shape
        q, s, qT, sT = o if o is not None else (None, None, None, None)
        q = _out(q, (n, k), E4M3, w.device)
        s = _out(s, (n // 128, k // 128), torch.float32, w.device)
        qT = _out(qT, (k, n), E4M3, w.device)
        sT = _out(sT, (k // 128, n // 128), torch.float32, w.device)
        descs[i] = WeightDesc(_ptr(w), n, k, w.stride(0), _ptr(q), _ptr(s), _ptr(qT), _ptr(sT))
        result.append((q, s, qT, sT))
    _run(dev, lib.fp8blk_quantize_weights_128x128_both, descs, len(weights), _stream_handle(stream, dev))
    return result


def fp8blk_amax_ema_workspace_bytes(rows: int) -> int:
    return int(lib.fp8blk_amax_ema_workspace_bytes(int(rows)))


def fp8blk_amax_ema(x, amax, scale=None, workspace=None, stream=None):
    """Per-tensor delayed scaling: update the amax buffer (float32 [1], in place) from max|x| by the
    EMA and write the tensor's scale.  Returns (amax, scale)."""
    x = _bf16_2d(x)
    dev = _need_cuda(x, amax, scale, workspace)
    if stream is not None and (scale is None or workspace is None):
        return _on_stream(stream, dev, lambda: fp8blk_amax_ema(x, amax, scale, workspace))
    rows, cols = x.shape
    if amax.dtype != torch.float32 or amax.numel() != 1:
        raise ValueError("amax must be a float32 tensor with one element")
    scale = _out(scale, (1,), torch.float32, x.device)
    need = fp8blk_amax_ema_workspace_bytes(rows)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _run(dev, lib.fp8blk_amax_ema, _ptr(x), rows, cols, x.stride(0), _ptr(amax), _ptr(scale), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    return amax, scale


AMAX_EMA_STATIC_MAX_ROWS = 65536   # FP8BLK_AMAX_EMA_STATIC_MAX_ROWS


def fp8blk_amax_ema_static(x, amax, scale, stream=None):
    """fp8blk_amax_ema with the library's own fixed scratch: allocates nothing (scale is required,
    float32 [1] on the device).  Calls on one device must be ordered; the first call on a device
    must come before graph capture.  Returns (amax, scale)."""
    x = _bf16_2d(x)
    if scale is None:
        raise ValueError("scale is required: this entry point allocates nothing")
    dev = _need_cuda(x, amax, scale)
    rows, cols = x.shape
    for t, name in ((amax, "amax"), (scale, "scale")):
        if t.dtype != torch.float32 or t.numel() != 1:
            raise ValueError(f"{name} must be a float32 tensor with one element")
    _run(dev, lib.fp8blk_amax_ema_static, _ptr(x), rows, cols, x.stride(0), _ptr(amax), _ptr(scale),
                                     _stream_handle(stream, dev))
    return amax, scale


def fp8blk_quantize_tensor(x, scale, q=None, stream=None):
    """The whole tensor with its one scale (device float32 [1]).  Returns q [rows, cols] E4M3."""
    x = _bf16_2d(x)
    dev = _need_cuda(x, _tensor_scale(scale), q)
    if stream is not None and q is None:
        return _on_stream(stream, dev, lambda: fp8blk_quantize_tensor(x, scale))
    rows, cols = x.shape
    q = _out(q, (rows, cols), E4M3, x.device)
    _run(dev, lib.fp8blk_quantize_tensor, _ptr(x), rows, cols, x.stride(0), _ptr(scale), _ptr(q), _stream_handle(stream, dev))
    return q


def fp8blk_gemm_tensor_scaled(a, sa, b, sb, d=None, stream=None):
    """D[M,N] = bf16(sa * sb * A . B^T) with one scale per E4M3 operand (device float32 [1] each)."""
    dev = _need_cuda(a, sa, b, sb, d)
    if stream is not None and d is None:
        return _on_stream(stream, dev, lambda: fp8blk_gemm_tensor_scaled(a, sa, b, sb))
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or a.dtype != E4M3 or b.dtype != E4M3:
        raise ValueError("A [M,K] and B [N,K] must be float8_e4m3fn")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("operands must be contiguous")
    _tensor_scale(sa), _tensor_scale(sb)
    if d is None:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    elif d.dtype != torch.bfloat16 or tuple(d.shape) != (m, n) or d.stride(1) != 1:
        raise ValueError("d must be a bfloat16 [M,N] tensor with unit column stride")
    _run(dev, lib.fp8blk_gemm_tensor_scaled, m, n, k, _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d), d.stride(0),
                                        _stream_handle(stream, dev))
    return d


def fp8_linear_delayed_forward(x, w, x_amax, w_amax, stream=None):
    """Y = X . W^T with per-tensor delayed scaling: both amax buffers updated by the EMA, both
    tensors quantised with their one scale, one GEMM.  Returns Y (bf16)."""
    if stream is not None:
        return _on_stream(stream, _need_cuda(x, w), lambda: fp8_linear_delayed_forward(x, w, x_amax, w_amax))
    _, sx = fp8blk_amax_ema(x, x_amax)
    _, sw = fp8blk_amax_ema(w, w_amax)
    qx = fp8blk_quantize_tensor(x, sx)
    qw = fp8blk_quantize_tensor(w, sw)
    return fp8blk_gemm_tensor_scaled(qx, sx, qw, sw)


def fp8blk_get_device_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error status code."""
    return int(lib.fp8blk_get_device_error(_stream_handle(stream)))


def fp8blk_version() -> int:
    return int(lib.fp8blk_version())


def linear_forward(x, w, stream=None):
    """Y = X . W^T through the FP8 blockwise path: quantise X (1x128) and W (128x128), then GEMM."""
    if stream is not None:
        return _on_stream(stream, _need_cuda(x, w), lambda: linear_forward(x, w))
    qx, sx, _, _ = fp8blk_quantize_act_1x128(x, ROWWISE)
    qw, sw = fp8blk_quantize_weight_128x128(w)
    return fp8blk_gemm(FWD, qx, sx, qw, sw)


def linear_backward(x, w, dy, stream=None):
    """(dX, dW) of Y = X . W^T: dX = dY . W (dgrad), dW = dY^T . X (wgrad), both FP8 blockwise."""
    if stream is not None:
        return _on_stream(stream, _need_cuda(x, w, dy), lambda: linear_backward(x, w, dy))
    qdy, sdy, qdyT, sdyT = fp8blk_quantize_act_1x128(dy, BOTH)
    qwT, swT = fp8blk_quantize_weight_128x128_t(w)
    _, _, qxT, sxT = fp8blk_quantize_act_1x128(x, COLWISE_T)
    dx = fp8blk_gemm(DGRAD, qdy, sdy, qwT, swT)
    dw = fp8blk_gemm(WGRAD, qdyT, sdyT, qxT, sxT)
    return dx, dw


def fp8blk_grouped_padded_rows(rows: int, groups: int) -> int:
    """Columns of the COLWISE_T outputs for `rows` rows in `groups` groups (whole 128-token blocks each)."""
    return int(lib.fp8blk_grouped_padded_rows(int(rows), int(groups)))


def _offsets(offsets) -> int:
    """Checks the offsets of rows sorted by group; returns the number of groups."""
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 tensor [groups + 1]")
    groups = offsets.numel() - 1
    if not 1 <= groups <= MAX_GROUPS:
        raise ValueError(f"between 1 and {MAX_GROUPS} groups")
    return groups


def fp8blk_quantize_act_1x128_grouped(x, offsets, mode=ROWWISE, q_row=None, s_row=None, q_colT=None, s_colT=None,
                                      stream=None):
    """Activation quantisation in 1x128 groups of rows sorted by group (offsets: int32 [groups + 1] on
    the device).  Any number of rows; groups of 128 tokens start anew in every group.  Returns (q_row,
    s_row, q_colT, s_colT); unused are None.  ``mode`` may include E5M2."""
    x = _bf16_2d(x)
    groups = _offsets(offsets)
    dev = _need_cuda(x, offsets, q_row, s_row, q_colT, s_colT)
    if stream is not None and _some_missing(mode, q_row, s_row, q_colT, s_colT):
        return _on_stream(stream, dev, lambda: fp8blk_quantize_act_1x128_grouped(x, offsets, mode, q_row, s_row, q_colT,
                                                                                 s_colT))
    rows, cols = x.shape
    code_dtype = E5M2_DTYPE if mode & E5M2 else E4M3
    if mode & ROWWISE:
        q_row = _out(q_row, (rows, cols), code_dtype, dev)
        s_row = _out(s_row, (cols // 128, rows), torch.float32, dev)
    else:
        q_row = s_row = None
    if mode & COLWISE_T:
        padded = fp8blk_grouped_padded_rows(rows, groups)
        q_colT = _out(q_colT, (cols, padded), code_dtype, dev)
        s_colT = _out(s_colT, (padded // 128, cols), torch.float32, dev)
    else:
        q_colT = s_colT = None
    _run(dev, lib.fp8blk_quantize_act_1x128_grouped, _ptr(x), rows, cols, _pitch(x, cols), int(mode),
         _ptr(offsets), groups, _ptr(q_row), _ptr(s_row), _ptr(q_colT), _ptr(s_colT), _stream_handle(stream, dev))
    return q_row, s_row, q_colT, s_colT


def fp8blk_gemm_grouped(layout, a, sa, b, sb, offsets, d=None, stream=None, out_dtype=torch.bfloat16):
    """The GEMM of a layer with one weight per group, over rows sorted by group (offsets: int32
    [groups + 1] on the device).  FWD: Y[T,out] from a[T,in], b[groups*out,in]; DGRAD: dX[T,in] from
    a[T,out], b[in,groups*out]; WGRAD: dW[groups,out,in] from a[out,P], b[in,P].  bf16, or fp32 with
    out_dtype=torch.float32 or an fp32 d.  Rows of d outside every group are left as they were."""
    groups = _offsets(offsets)
    dev = _need_cuda(a, sa, b, sb, offsets, d)
    if stream is not None and d is None:
        return _on_stream(stream, dev,
                          lambda: fp8blk_gemm_grouped(layout, a, sa, b, sb, offsets, out_dtype=out_dtype))
    if a.dim() != 2 or b.dim() != 2 or a.dtype not in (E4M3, E5M2_DTYPE) or b.dtype not in (E4M3, E5M2_DTYPE):
        raise ValueError("A and B must be 2-D float8_e4m3fn or float8_e5m2")
    m, k = a.shape
    if layout == WGRAD:
        n = b.shape[0]
        want_b, want_sb, shape = (n, k), (k // 128, n), (groups, m, n)
    elif layout == FWD:
        n = b.shape[0] // groups
        want_b, want_sb, shape = (groups * n, k), (groups * n // 128, k // 128), (m, n)
    elif layout == DGRAD:
        n = b.shape[0]
        want_b, want_sb, shape = (n, groups * k), (n // 128, groups * k // 128), (m, n)
    else:
        raise ValueError("layout must be FWD, DGRAD or WGRAD")
    if tuple(b.shape) != want_b:
        raise ValueError(f"B {tuple(b.shape)} does not match A {tuple(a.shape)} and {groups} groups")
    if tuple(sa.shape) != (k // 128, m) or tuple(sb.shape) != want_sb:
        raise ValueError(f"scale shapes {tuple(sa.shape)}, {tuple(sb.shape)} do not match layout {layout}")
    if sa.dtype != torch.float32 or sb.dtype != torch.float32:
        raise ValueError("scales must be float32")
    if not (a.is_contiguous() and b.is_contiguous() and sa.is_contiguous() and sb.is_contiguous()):
        raise ValueError("operands and scales must be contiguous")
    if d is None:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        d = _empty(shape, out_dtype, dev)
    elif d.dtype not in (torch.bfloat16, torch.float32) or tuple(d.shape) != shape or d.stride(-1) != 1 or (
            layout == WGRAD and groups > 1 and d.stride(0) != m * d.stride(1)):
        raise ValueError(f"d must be a bfloat16 or float32 {shape} tensor with unit column stride and one row pitch")
    flags = (A_E5M2 if a.dtype == E5M2_DTYPE else 0) | (B_E5M2 if b.dtype == E5M2_DTYPE else 0)
    flags |= OUT_F32 if d.dtype == torch.float32 else 0
    _run(dev, lib.fp8blk_gemm_grouped, int(layout) | flags, groups, _ptr(offsets), m, n, k, _ptr(a), _ptr(sa), _ptr(b),
         _ptr(sb), _ptr(d), d.stride(-2) if layout == WGRAD else _pitch(d, n), _stream_handle(stream, dev))
    return d


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(size, *args) -> int:
    """size(*args), remembered: the library's answer depends on nothing else, and asking costs a call of it."""
    return size(*args)


def fp8blk_linear_grouped_workspace_bytes(groups: int, rows: int, k: int) -> int:
    """Bytes of workspace fp8blk_linear_grouped needs for x [rows, k] in `groups` groups (0: none)."""
    return int(lib.fp8blk_linear_grouped_workspace_bytes(int(groups), int(rows), int(k)))


def fp8blk_linear_grouped(x, qw, sw, offsets, d=None, workspace=None, stream=None, out_dtype=torch.bfloat16):
    """Y[t] = X[t] . W[e]^T for the rows t of group e, x [T,in] bf16 quantised on the way, W [groups,out,in]
    ahead as one weight of groups*out rows (qw, sw): the result of fp8blk_quantize_act_1x128_grouped and
    fp8blk_gemm_grouped, in one launch with up to 16 rows.  workspace: a uint8 CUDA tensor of at least
    fp8blk_linear_grouped_workspace_bytes(groups, T, in) bytes (allocated here when None and needed)."""
    x = _bf16_2d(x)
    groups = _offsets(offsets)
    dev = _need_cuda(x, qw, sw, offsets, d, workspace)
    if stream is not None and (d is None or workspace is None):
        return _on_stream(stream, dev,
                          lambda: fp8blk_linear_grouped(x, qw, sw, offsets, d, workspace, None, out_dtype))
    rows, k = x.shape
    n = qw.shape[0] // groups
    if qw.dtype != E4M3 or sw.dtype != torch.float32:
        raise ValueError("the weight's codes are float8_e4m3fn and its scales float32")
    if tuple(qw.shape) != (groups * n, k) or tuple(sw.shape) != (groups * n // 128, k // 128):
        raise ValueError(f"weight {tuple(qw.shape)}, {tuple(sw.shape)} does not match X {tuple(x.shape)} and {groups} groups")
    if not (qw.is_contiguous() and sw.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    if workspace is None:
        need = _workspace_bytes(fp8blk_linear_grouped_workspace_bytes, groups, rows, k)
        if need > 0:                           # else one launch, which needs none
            workspace = _empty((need,), torch.uint8, dev)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    if d is None:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        d = _empty((rows, n), out_dtype, dev)
    elif d.dtype not in (torch.bfloat16, torch.float32) or tuple(d.shape) != (rows, n) or d.stride(1) != 1:
        raise ValueError(f"d must be a bfloat16 or float32 {(rows, n)} tensor with unit column stride")
    pitch, ldx = _pitch(d, n), _pitch(x, k)
    _run(dev, lib.fp8blk_linear_grouped, OUT_F32 if d.dtype == torch.float32 else 0, groups, offsets.data_ptr(), rows, n,
         k, x.data_ptr(), ldx, qw.data_ptr(), sw.data_ptr(), _ptr(workspace), 0 if workspace is None else workspace.numel(),
         d.data_ptr(), pitch,
         _stream_handle(stream, dev))
    return d


def grouped_linear_forward(x, qw, sw, offsets, stream=None):
    """Y[t] = X[t] . W[e]^T for the rows t of group e: X quantised here (1x128), W [groups,out,in] ahead, as
    one weight of groups*out rows (fp8blk_quantize_weight_128x128: qw [groups*out,in], sw)."""
    return fp8blk_linear_grouped(x, qw, sw, offsets, stream=stream)


def grouped_linear_backward(x, dy, qwT, swT, offsets, stream=None, out_dtype=torch.bfloat16):
    """(dX [T,in], dW [groups,out,in]) of grouped_linear_forward, both FP8 blockwise; the transposed weights
    come quantised (fp8blk_quantize_weight_128x128_t or _both: qwT [in,groups*out], swT).  out_dtype: dW's."""
    _same_tokens(x, dy)
    if stream is not None:
        return _on_stream(stream, _need_cuda(x, dy),
                          lambda: grouped_linear_backward(x, dy, qwT, swT, offsets, None, out_dtype))
    qdy, sdy, qdyT, sdyT = fp8blk_quantize_act_1x128_grouped(dy, offsets, BOTH)
    _, _, qxT, sxT = fp8blk_quantize_act_1x128_grouped(x, offsets, COLWISE_T)
    dx = fp8blk_gemm_grouped(DGRAD, qdy, sdy, qwT, swT, offsets)
    dw = fp8blk_gemm_grouped(WGRAD, qdyT, sdyT, qxT, sxT, offsets, out_dtype=out_dtype)
    return dx, dw


MX4_BLOCK = {MXFP4: 32, NVFP4: 16}


def fp8blk_mx4_scale_bytes(fmt, rows: int, k: int) -> int:
    """Bytes of the scales of a [rows, k] operand in a 4-bit format."""
    return int(lib.fp8blk_mx4_scale_bytes(int(fmt), int(rows), int(k)))


def _mx4_scale_shape(fmt, rows: int, k: int) -> tuple:
    return -(-rows // 128), -(-k // (4 * MX4_BLOCK[fmt])), 512


def _tensor_scale(t):
    if t is not None and (t.dtype != torch.float32 or t.numel() != 1):
        raise ValueError("a tensor scale is a float32 tensor with one element")
    return t


def _mx4_operand(q, s, fmt, name) -> tuple:
    """(rows, k) of a 4-bit operand."""
    if q.dtype != torch.uint8 or q.dim() != 2 or s.dtype != torch.uint8:
        raise ValueError(f"{name}: codes [rows, k/2] and scales are uint8")
    rows, k = q.shape[0], 2 * q.shape[1]
    if tuple(s.shape) != _mx4_scale_shape(fmt, rows, k):
        raise ValueError(f"{name}: scales must have shape {_mx4_scale_shape(fmt, rows, k)}")
    if not (q.is_contiguous() and s.is_contiguous()):
        raise ValueError(f"{name}: codes and scales must be contiguous")
    return rows, k


def fp8blk_quantize_mx4(x, fmt, mode=ROWWISE, tensor_scale=None, q_row=None, s_row=None, q_colT=None, s_colT=None,
                        stream=None):
    """4-bit quantisation of a [R,C] bf16 tensor.  fmt: MXFP4 or NVFP4 (tensor_scale: float32 [1] on the
    device).  Returns (q_row, s_row, q_colT, s_colT); unused are None."""
    x = _bf16_2d(x)
    if fmt not in MX4_BLOCK:
        raise ValueError("fmt must be MXFP4 or NVFP4")
    dev = _need_cuda(x, _tensor_scale(tensor_scale), q_row, s_row, q_colT, s_colT)
    if stream is not None and _some_missing(mode, q_row, s_row, q_colT, s_colT):
        return _on_stream(stream, dev,
                          lambda: fp8blk_quantize_mx4(x, fmt, mode, tensor_scale, q_row, s_row, q_colT, s_colT))
    rows, cols = x.shape
    if mode & ROWWISE:
        q_row = _out(q_row, (rows, cols // 2), torch.uint8, dev)
        s_row = _out(s_row, _mx4_scale_shape(fmt, rows, cols), torch.uint8, dev)
    else:
        q_row = s_row = None
    if mode & COLWISE_T:
        padded = -(-rows // 32) * 32
        q_colT = _out(q_colT, (cols, padded // 2), torch.uint8, dev)
        s_colT = _out(s_colT, _mx4_scale_shape(fmt, cols, padded), torch.uint8, dev)
    else:
        q_colT = s_colT = None
    _run(dev, lib.fp8blk_quantize_mx4, _ptr(x), rows, cols, _pitch(x, cols), int(mode),
         int(fmt), _ptr(tensor_scale), _ptr(q_row), _ptr(s_row), _ptr(q_colT), _ptr(s_colT),
         _stream_handle(stream, dev))
    return q_row, s_row, q_colT, s_colT


def fp8blk_dequantize_mx4(q, s, fmt, tensor_scale=None, y=None, stream=None):
    """The bf16 values [R,C] of codes q [R,C/2] and scales s of fp8blk_quantize_mx4."""
    if fmt not in MX4_BLOCK:
        raise ValueError("fmt must be MXFP4 or NVFP4")
    dev = _need_cuda(q, s, _tensor_scale(tensor_scale), y)
    if stream is not None and y is None:
        return _on_stream(stream, dev, lambda: fp8blk_dequantize_mx4(q, s, fmt, tensor_scale))
    rows, cols = _mx4_operand(q, s, fmt, "q")
    if y is None:
        y = _empty((rows, cols), torch.bfloat16, dev)
    elif y.dtype != torch.bfloat16 or tuple(y.shape) != (rows, cols) or y.stride(1) != 1:
        raise ValueError(f"y must be a bfloat16 tensor of shape {(rows, cols)} with unit column stride")
    _run(dev, lib.fp8blk_dequantize_mx4, _ptr(q), _ptr(s), rows, cols, int(fmt), _ptr(tensor_scale), _ptr(y),
         _pitch(y, cols), _stream_handle(stream, dev))
    return y


def fp8blk_gemm_mx4(a, sa, b, sb, fmt, tensor_sa=None, tensor_sb=None, d=None, stream=None, out_dtype=torch.bfloat16):
    """D[M,N] of 4-bit operands a [M,K/2] and b [N,K/2] (fp8blk_quantize_mx4), accumulated in fp32; bf16, or
    fp32 with out_dtype=torch.float32 or an fp32 d.  A d made here has rows of a multiple of 8 elements."""
    if fmt not in MX4_BLOCK:
        raise ValueError("fmt must be MXFP4 or NVFP4")
    dev = _need_cuda(a, sa, b, sb, _tensor_scale(tensor_sa), _tensor_scale(tensor_sb), d)
    if stream is not None and d is None:
        return _on_stream(stream, dev,
                          lambda: fp8blk_gemm_mx4(a, sa, b, sb, fmt, tensor_sa, tensor_sb, out_dtype=out_dtype))
    m, k = _mx4_operand(a, sa, fmt, "A")
    n, kb = _mx4_operand(b, sb, fmt, "B")
    if k != kb:
        raise ValueError("A and B disagree on K")
    if d is None:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        pitch = -(-n // 8) * 8
        d = _empty((m, pitch), out_dtype, dev)
        if pitch != n:
            d = d[:, :n]
    elif d.dtype not in (torch.bfloat16, torch.float32) or tuple(d.shape) != (m, n) or d.stride(1) != 1:
        raise ValueError("d must be a bfloat16 or float32 [M,N] tensor with unit column stride")
    pitch = _pitch(d, n)
    _run(dev, lib.fp8blk_gemm_mx4, int(fmt) | (OUT_F32 if d.dtype == torch.float32 else 0), m, n, k, _ptr(a), _ptr(sa),
         _ptr(tensor_sa), _ptr(b), _ptr(sb), _ptr(tensor_sb), _ptr(d), pitch, _stream_handle(stream, dev))
    return d


def fp8blk_linear_mx4_workspace_bytes(fmt, m: int, k: int) -> int:
    """Bytes of workspace fp8blk_linear_mx4 needs for x [m, k] (0 for m <= 16)."""
    return int(lib.fp8blk_linear_mx4_workspace_bytes(int(fmt), int(m), int(k)))


def fp8blk_linear_mx4(x, qw, sw, fmt, tensor_sx=None, tensor_sw=None, d=None, workspace=None, stream=None,
                      out_dtype=torch.bfloat16):
    """Y = X . W^T in 4 bits, x [M,K] bf16 quantised on the way, W [N,K] ahead (qw [N,K/2], sw): the result of
    fp8blk_quantize_mx4 and fp8blk_gemm_mx4, in one launch when M <= 16.  workspace: a uint8 CUDA tensor of at
    least fp8blk_linear_mx4_workspace_bytes(fmt, M, K) bytes (allocated here when None and needed)."""
    x = _bf16_2d(x)
    if fmt not in MX4_BLOCK:
        raise ValueError("fmt must be MXFP4 or NVFP4")
    dev = _need_cuda(x, qw, sw, _tensor_scale(tensor_sx), _tensor_scale(tensor_sw), d, workspace)
    n, k = _mx4_operand(qw, sw, fmt, "W")
    if stream is not None and (d is None or workspace is None):
        return _on_stream(stream, dev, lambda: fp8blk_linear_mx4(x, qw, sw, fmt, tensor_sx, tensor_sw, d, workspace,
                                                                 None, out_dtype))
    m = x.shape[0]
    if x.shape[1] != k:
        raise ValueError("X and W disagree on their features")
    if workspace is None:
        need = _workspace_bytes(fp8blk_linear_mx4_workspace_bytes, fmt, m, k)
        if need > 0:                           # else one launch, which needs none
            workspace = _empty((need,), torch.uint8, dev)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    if d is None:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        pitch = -(-n // 8) * 8
        d = _empty((m, pitch), out_dtype, dev)
        if pitch != n:
            d = d[:, :n]
    elif d.dtype not in (torch.bfloat16, torch.float32) or tuple(d.shape) != (m, n) or d.stride(1) != 1:
        raise ValueError("d must be a bfloat16 or float32 [M,N] tensor with unit column stride")
    pitch, ldx = _pitch(d, n), _pitch(x, k)
    _run(dev, lib.fp8blk_linear_mx4, fmt | (OUT_F32 if d.dtype == torch.float32 else 0), m, n, k, x.data_ptr(), ldx,
         _ptr(tensor_sx), qw.data_ptr(), sw.data_ptr(), _ptr(tensor_sw), _ptr(workspace),
         0 if workspace is None else workspace.numel(), d.data_ptr(), pitch, _stream_handle(stream, dev))
    return d


def mx4_linear_forward(x, qw, sw, fmt, x_scale=None, w_scale=None, stream=None):
    """Y = X . W^T in 4 bits: X quantised here, W [out,in] ahead (fp8blk_quantize_mx4, ROWWISE)."""
    return fp8blk_linear_mx4(x, qw, sw, fmt, x_scale, w_scale, stream=stream)


def mx4_linear_wgrad(x, dy, fmt, x_scale=None, dy_scale=None, stream=None, out_dtype=torch.bfloat16):
    """dW = dY^T . X in 4 bits, both quantised here along the tokens."""
    # The calls of fp8blk_quantize_mx4 (COLWISE_T, twice) and fp8blk_gemm_mx4 with one allocation for the codes
    # and scales between them: with few tokens the host's time is what counts.
    x, dy = _bf16_2d(x), _bf16_2d(dy)
    _same_tokens(x, dy)
    if fmt not in MX4_BLOCK:
        raise ValueError("fmt must be MXFP4 or NVFP4")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    dev = _need_cuda(x, dy, _tensor_scale(x_scale), _tensor_scale(dy_scale))
    if stream is not None:
        return _on_stream(stream, dev, lambda: mx4_linear_wgrad(x, dy, fmt, x_scale, dy_scale, None, out_dtype))
    tokens, k = x.shape
    n = dy.shape[1]
    padded = -(-tokens // 32) * 32
    at, places = 0, []                     # codes and scales of dY, then of X, all on 16-byte boundaries
    for rows in (n, k):
        blocks, atoms, size = _mx4_scale_shape(fmt, rows, padded)
        places += [at, at + rows * padded // 2]
        at = places[-1] + blocks * atoms * size
    work = _empty((at,), torch.uint8, dev)
    pitch = -(-k // 8) * 8
    dw = _empty((n, pitch), out_dtype, dev)
    base, handle, gx, gd = work.data_ptr(), _stream_handle(None, dev), _ptr(x_scale), _ptr(dy_scale)
    qd, sd, qx, sx = (base + p for p in places) if tokens else (None,) * 4
    _run(dev, lib.fp8blk_quantize_mx4, dy.data_ptr(), tokens, n, _pitch(dy, n), COLWISE_T, fmt, gd, None, None, qd, sd, handle)
    _run(dev, lib.fp8blk_quantize_mx4, x.data_ptr(), tokens, k, _pitch(x, k), COLWISE_T, fmt, gx, None, None, qx, sx, handle)
    _run(dev, lib.fp8blk_gemm_mx4, fmt | (OUT_F32 if out_dtype == torch.float32 else 0), n, k, padded, qd, sd, gd, qx, sx,
         gx, dw.data_ptr(), pitch, handle)
    return dw if pitch == k else dw[:, :k]


def mx4_linear_backward(x, dy, qwT, swT, fmt, x_scale=None, dy_scale=None, w_scale=None, stream=None,
                        out_dtype=torch.bfloat16):
    """(dX, dW) of Y = X . W^T in 4 bits: dY quantised once along features and along tokens, X along
    tokens, W ahead (fp8blk_quantize_mx4, COLWISE_T).  out_dtype: dW's."""
    _same_tokens(x, dy)
    if stream is not None:
        return _on_stream(stream, _need_cuda(x, dy), lambda: mx4_linear_backward(x, dy, qwT, swT, fmt, x_scale, dy_scale,
                                                                                 w_scale, None, out_dtype))
    qd, sd, qdT, sdT = fp8blk_quantize_mx4(dy, fmt, BOTH, dy_scale)
    _, _, qxT, sxT = fp8blk_quantize_mx4(x, fmt, COLWISE_T, x_scale)
    dx = fp8blk_gemm_mx4(qd, sd, qwT, swT, fmt, dy_scale, w_scale)
    dw = fp8blk_gemm_mx4(qdT, sdT, qxT, sxT, fmt, dy_scale, x_scale, out_dtype=out_dtype)
    return dx, dw
