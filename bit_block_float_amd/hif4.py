"""Python binding of libhif4.so (the C ABI in include/hif4.h).

Argument marshalling only: every step runs in the library's HIP kernels.
PyTorch provides device memory and the current HIP stream. There is no CPU
fallback: if the library or a gfx950 device is missing, calls raise.

Tensors: bf16 inputs are torch.bfloat16 on the GPU; codes are uint8
[rows][k/2]; meta is int32 [rows][k/64] holding the u32 metadata words bit
for bit; masks are uint8.
"""
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhif4.so")

HIF4_F32, HIF4_BF16 = 0, 1
_lib = None


class Hif4Error(RuntimeError):
    def __init__(self, status, what):
        super().__init__(f"{what}: {lib().hif4_status_string(status).decode()} (status {status})")
        self.status = status


def lib():
    """The loaded library (ctypes). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m bit_block_float_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        p, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        L.hif4_status_string.argtypes = [ctypes.c_int]
        L.hif4_status_string.restype = ctypes.c_char_p
        L.hif4_version.argtypes = []
        L.hif4_version.restype = ctypes.c_int
        L.hif4_quantize.argtypes = [p, i64, i64, i64, p, i64, p, p, p, p]
        L.hif4_quantize.restype = ctypes.c_int
        L.hif4_dequantize.argtypes = [p, p, i64, i64, p, ctypes.c_int, p]
        L.hif4_dequantize.restype = ctypes.c_int
        L.hif4_linear_workspace_bytes.argtypes = [i64, i64, i64, i64]
        L.hif4_linear_workspace_bytes.restype = sz
        L.hif4_linear_w4a4.argtypes = [p, p, p, p, p, p, p, p, i64, i64, i64, i64, p, ctypes.c_int,
                                       p, sz, p]
        L.hif4_linear_w4a4.restype = ctypes.c_int
        L.hif4_linear_xcodes_wbf16.argtypes = [p, p, p, p, p, i64, i64, i64, i64, p, ctypes.c_int, p,
                                               sz, p]
        L.hif4_linear_xcodes_wbf16.restype = ctypes.c_int
        L.hif4_linear_xcodes_wbf16_noalloc.argtypes = [p, p, p, p, p, i64, i64, i64, i64, p,
                                                       ctypes.c_int, p]
        L.hif4_linear_xcodes_wbf16_noalloc.restype = ctypes.c_int
        L.hif4_percentile_workspace_bytes.argtypes = [i64, i64]
        L.hif4_percentile_workspace_bytes.restype = sz
        L.hif4_percentile_mask.argtypes = [p, i64, i64, i64, ctypes.c_double, i64, p, p, p, sz, p]
        L.hif4_percentile_mask.restype = ctypes.c_int
        L.hif4_quantize_f32.argtypes = [p, i64, i64, i64, p, p, p]
        L.hif4_quantize_offsets.argtypes = [p, i64, i64, i64, p, p, p, p, p]
        L.hif4_quantize_offsets.restype = ctypes.c_int
        L.hif4_quantize_f32.restype = ctypes.c_int
        L.hif4_higptq_workspace_bytes.argtypes = [i64]
        L.hif4_higptq_workspace_bytes.restype = sz
        L.hif4_higptq_unit.argtypes = [p, i64, i64, i64, p, i64, i64, ctypes.c_int, p, p, p, sz, p]
        L.hif4_higptq_unit.restype = ctypes.c_int
        L.hif4_higptq_block_workspace_bytes.argtypes = [i64, i64]
        L.hif4_higptq_block_workspace_bytes.restype = sz
        L.hif4_higptq_block.argtypes = [p, i64, i64, i64, p, i64, i64, i64, ctypes.c_int, p, p, p,
                                        sz, p]
        L.hif4_higptq_block.restype = ctypes.c_int
        i, d = ctypes.c_int, ctypes.c_double
        L.hif4_quantize_fp8.argtypes = [p, i, i64, i64, i64, i64, i, p, p, i64, p]
        L.hif4_quantize_fp8.restype = i
        L.hif4_quantize_fp8_both.argtypes = [p, i, i64, i64, i64, i64, p, p, i64, p, p, i64, p]
        L.hif4_quantize_fp8_both.restype = i
        L.hif4_dequantize_fp8.argtypes = [p, p, i, i64, i64, i64, i64, p, i, p]
        L.hif4_dequantize_fp8.restype = i
        L.hif4_linear_fp8_workspace_bytes.argtypes = [i64, i64, i64]
        L.hif4_linear_fp8_workspace_bytes.restype = sz
        L.hif4_linear_fp8.argtypes = [p, p, i64, p, p, i64, i, i64, i64, i64, i64, p, i, p, sz, p]
        L.hif4_linear_fp8.restype = i
        L.hif4_linear_fp8_backward_workspace_bytes.argtypes = [i64, i64, i64]
        L.hif4_linear_fp8_backward_workspace_bytes.restype = sz
        L.hif4_linear_fp8_backward.argtypes = [p, i, i64, p, p, i64, p, p, i64, i, i64, i64, i64, i64,
                                               p, i, p, i, p, sz, p]
        L.hif4_linear_fp8_backward.restype = i
        L.hif4_mxfp4_columns.argtypes = [i64, i64]
        L.hif4_mxfp4_columns.restype = i64
        L.hif4_quantize_mxfp4.argtypes = [p, i, i64, i64, i64, i64, i, p, i64, p, p, p]
        L.hif4_quantize_mxfp4.restype = i
        L.hif4_quantize_mxfp4_both.argtypes = [p, i, i64, i64, i64, i64, p, i64, p, p, p, p, p]
        L.hif4_quantize_mxfp4_both.restype = i
        L.hif4_dequantize_mxfp4.argtypes = [p, p, i64, i64, p, i, p]
        L.hif4_dequantize_mxfp4.restype = i
        L.hif4_linear_mxfp4_workspace_bytes.argtypes = [i64, i64, i64]
        L.hif4_linear_mxfp4_workspace_bytes.restype = sz
        L.hif4_linear_mxfp4.argtypes = [p, p, p, p, i64, i64, i64, p, i, p, sz, p]
        L.hif4_linear_mxfp4.restype = i
        L.hif4_linear_mxfp4_grouped.argtypes = [p, p, p, p, p, i64, i64, i64, i64, p, i, p]
        L.hif4_linear_mxfp4_grouped.restype = i
        L.hif4_linear_mxfp4_backward_workspace_bytes.argtypes = [i64, i64, i64]
        L.hif4_linear_mxfp4_backward_workspace_bytes.restype = sz
        L.hif4_linear_mxfp4_backward.argtypes = [p, i, i64, p, p, p, p, i64, i64, i64, p, i, p, i, p, sz, p]
        L.hif4_linear_mxfp4_backward.restype = i
        L.hif4_linear_mxfp4_grouped_backward_workspace_bytes.argtypes = [i64, i64, i64, i64]
        L.hif4_linear_mxfp4_grouped_backward_workspace_bytes.restype = sz
        L.hif4_linear_mxfp4_grouped_backward.argtypes = [p, i, i64, p, p, p, p, p, i64, i64, i64, i64, p, i, p,
                                                         i, p, sz, p]
        L.hif4_linear_mxfp4_grouped_backward.restype = i
        L.hif4_layer_norm.argtypes = [p, i, i64, i64, i64, p, p, i, d, p, i64, p, p, p]
        L.hif4_layer_norm.restype = i
        L.hif4_layer_norm_quantize.argtypes = [p, i, i64, i64, i64, p, p, i, d, p, i64, p, p, p, p]
        L.hif4_layer_norm_quantize.restype = i
        L.hif4_layer_norm_quantize_fp8.argtypes = [p, i, i64, i64, i64, p, p, i, d, p, p, i64, p]
        L.hif4_layer_norm_quantize_fp8.restype = i
        L.hif4_layer_norm_quantize_mxfp4.argtypes = [p, i, i64, i64, i64, p, p, i, d, p, p, p]
        L.hif4_layer_norm_quantize_mxfp4.restype = i
        L.hif4_layer_norm_backward_workspace_bytes.argtypes = [i64, i64]
        L.hif4_layer_norm_backward_workspace_bytes.restype = sz
        L.hif4_layer_norm_backward.argtypes = [p, i64, p, i64, i, i64, i64, p, p, p, i, p, i64, p, p,
                                               p, sz, p]
        L.hif4_layer_norm_backward.restype = i
        _lib = L
    return _lib


def require_gpu():
    """Raise unless a gfx950 GPU is visible and the library loads."""
    lib()
    if not torch.cuda.is_available():
        raise RuntimeError("no GPU visible: libhif4 runs only on gfx950 (MI355X)")
    arch = torch.cuda.get_device_properties(torch.cuda.current_device()).gcnArchName
    if not arch.startswith("gfx950"):
        raise RuntimeError(f"libhif4 needs gfx950, found {arch}")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ok(status, what):
    if status != 0:
        raise Hif4Error(status, what)


def _check_bf16_rows(x, name):
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D bf16 CUDA tensor with unit column stride")


def quantize(x, mask=None, codes=None, meta=None, kept=None, stream=None):
    """HiF4-quantize bf16 x [rows][k] along k -> (codes u8, meta int32, kept bf16)."""
    _check_bf16_rows(x, "x")
    rows, k = x.shape
    dev = x.device
    codes = codes if codes is not None else torch.empty((rows, k // 2), dtype=torch.uint8, device=dev)
    meta = meta if meta is not None else torch.empty((rows, k // 64), dtype=torch.int32, device=dev)
    n_mask = 0
    if mask is not None:
        n_mask = int(torch.count_nonzero(mask).item())
        if kept is None:
            kept = torch.empty((rows, n_mask), dtype=torch.bfloat16, device=dev)
    st = lib().hif4_quantize(_ptr(x), rows, k, x.stride(0), _ptr(mask), n_mask,
                             _ptr(kept) if n_mask else None, _ptr(codes), _ptr(meta), _stream(stream))
    _ok(st, "hif4_quantize")
    return codes, meta, kept


def dequantize(codes, meta, out_dtype=torch.float32, out=None, stream=None):
    """Decode codes [rows][k/2] + meta [rows][k/64] -> [rows][k] fp32 or bf16."""
    rows, k = codes.shape[0], codes.shape[1] * 2
    dt = HIF4_F32 if out_dtype == torch.float32 else HIF4_BF16
    out = out if out is not None else torch.empty((rows, k), dtype=out_dtype, device=codes.device)
    st = lib().hif4_dequantize(_ptr(codes), _ptr(meta), rows, k, _ptr(out), dt, _stream(stream))
    _ok(st, "hif4_dequantize")
    return out


def linear_workspace_bytes(m, n, k, n_kept=0):
    return int(lib().hif4_linear_workspace_bytes(m, n, k, n_kept))


def _kept_count(x_kept, w_kept, m, n):
    """n_kept from the kept-value tensors, after checking their shapes: a
    short tensor would be read past its end by the library."""
    if w_kept is None:
        if x_kept is not None:
            raise ValueError("x_kept given without w_kept")
        return 0
    if (w_kept.dtype != torch.bfloat16 or not w_kept.is_contiguous() or w_kept.dim() != 2
            or w_kept.shape[0] != n or not w_kept.is_cuda):
        raise ValueError(f"w_kept must be a contiguous bf16 CUDA tensor [n={n}][n_kept]")
    if x_kept is not None and (x_kept.dtype != torch.bfloat16 or not x_kept.is_contiguous()
                               or x_kept.dim() != 2 or x_kept.shape[0] != m
                               or x_kept.shape[1] != w_kept.shape[1] or not x_kept.is_cuda):
        raise ValueError(f"x_kept must be a contiguous bf16 CUDA tensor [m={m}][n_kept]")
    return w_kept.shape[1]


def _check_mask(mask, k, n_kept):
    """The protection mask: uint8 [k] on the GPU with exactly n_kept nonzeros
    (the count the kept values were gathered for)."""
    if mask is None:
        if n_kept:
            raise ValueError("n_kept > 0 with a bf16 x needs the mask that selects the channels")
        return
    if mask.dtype != torch.uint8 or mask.shape != (k,) or not mask.is_contiguous() or not mask.is_cuda:
        raise ValueError(f"mask must be a contiguous uint8 CUDA tensor [k={k}]")
    nz = int(torch.count_nonzero(mask).item())
    if nz != n_kept:
        raise ValueError(f"mask has {nz} protected channels but the kept values have {n_kept}")


def linear_w4a4(w_codes, w_meta, x=None, x_codes=None, x_meta=None, mask=None, x_kept=None,
                w_kept=None, y_dtype=torch.float32, y=None, workspace=None, stream=None):
    """Y = deq(Q(X)) deq(Q(W))^T (+ x_kept w_kept^T over protected channels).
    X as bf16 x [m][k] (with `mask` when there are protected channels) or as
    (x_codes, x_meta[, x_kept])."""
    n, k = w_codes.shape[0], w_codes.shape[1] * 2
    if x is not None:
        _check_bf16_rows(x, "x")
        if not x.is_contiguous():
            raise ValueError("x must be contiguous (row stride k)")
        m = x.shape[0]
    else:
        m = x_codes.shape[0]
    n_kept = _kept_count(x_kept, w_kept, m, n)
    if x is not None:
        _check_mask(mask, k, n_kept)
    elif n_kept and x_kept is None:
        raise ValueError("X given as codes with protected channels needs x_kept")
    dev = w_codes.device
    dt = HIF4_F32 if y_dtype == torch.float32 else HIF4_BF16
    y = y if y is not None else torch.empty((m, n), dtype=y_dtype, device=dev)
    need = linear_workspace_bytes(m, n, k, n_kept)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    st = lib().hif4_linear_w4a4(_ptr(x), _ptr(x_codes), _ptr(x_meta), _ptr(w_codes), _ptr(w_meta),
                                _ptr(mask), _ptr(x_kept), _ptr(w_kept), n_kept, m, n, k, _ptr(y),
                                dt, _ptr(workspace), workspace.numel(), _stream(stream))
    _ok(st, "hif4_linear_w4a4")
    return y


def linear_xcodes_wbf16(x_codes, x_meta, w, x_kept=None, w_kept=None, y_dtype=torch.float32,
                        y=None, workspace=None, stream=None):
    """Y = deq(X codes) w^T (+ x_kept w_kept^T) with w bf16 [n][k] (e.g. a
    weight decoded once)."""
    _check_bf16_rows(w, "w")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous (row stride k)")
    m, n, k = x_codes.shape[0], w.shape[0], w.shape[1]
    n_kept = _kept_count(x_kept, w_kept, m, n)
    if n_kept and x_kept is None:
        raise ValueError("protected channels need x_kept")
    dt = HIF4_F32 if y_dtype == torch.float32 else HIF4_BF16
    y = y if y is not None else torch.empty((m, n), dtype=y_dtype, device=w.device)
    if workspace is None and n_kept:
        workspace = torch.empty((linear_workspace_bytes(m, n, 0, n_kept),), dtype=torch.uint8,
                                device=w.device)
    ws_bytes = workspace.numel() if workspace is not None else 0
    st = lib().hif4_linear_xcodes_wbf16(_ptr(x_codes), _ptr(x_meta), _ptr(w), _ptr(x_kept),
                                        _ptr(w_kept), n_kept, m, n, k, _ptr(y), dt,
                                        _ptr(workspace), ws_bytes, _stream(stream))
    _ok(st, "hif4_linear_xcodes_wbf16")
    return y


NOALLOC_SCRATCH_BYTES = 32 << 20  # HIF4_NOALLOC_SCRATCH_BYTES


def linear_xcodes_wbf16_noalloc(x_codes, x_meta, w, y, x_kept=None, w_kept=None, stream=None):
    """hif4_linear_xcodes_wbf16 without a workspace (the library's static
    scratch holds the protected-channel operands): Y into the caller's `y`
    ([m][n], fp32 or bf16). Allocates no device memory."""
    _check_bf16_rows(w, "w")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous (row stride k)")
    m, n, k = x_codes.shape[0], w.shape[0], w.shape[1]
    if y.shape != (m, n) or not y.is_contiguous() or y.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("y must be a contiguous fp32 or bf16 tensor [m][n]")
    n_kept = _kept_count(x_kept, w_kept, m, n)
    if n_kept and x_kept is None:
        raise ValueError("protected channels need x_kept")
    dt = HIF4_F32 if y.dtype == torch.float32 else HIF4_BF16
    st = lib().hif4_linear_xcodes_wbf16_noalloc(_ptr(x_codes), _ptr(x_meta), _ptr(w),
                                                _ptr(x_kept), _ptr(w_kept), n_kept, m, n, k,
                                                _ptr(y), dt, _stream(stream))
    _ok(st, "hif4_linear_xcodes_wbf16_noalloc")
    return y


def percentile_workspace_bytes(rows, c):
    return int(lib().hif4_percentile_workspace_bytes(rows, c))


def percentile_exact_channels(workspace, rows, c):
    """Channels of the last hif4_percentile_mask call on `workspace` whose
    statistic came from the two exact passes (c unless the one-pass window
    path ran; then the channels it missed). Reads the count from the device."""
    off = percentile_workspace_bytes(rows, c) - 256
    return int(workspace[off:off + 4].view(torch.int32).item())


def percentile_mask(x, q, n_protect, stats=None, mask=None, workspace=None, stream=None):
    """Per-channel type-7 quantile of |x| over rows -> (stats fp32 [c], mask u8 [c])."""
    _check_bf16_rows(x, "x")
    rows, c = x.shape
    dev = x.device
    stats = stats if stats is not None else torch.empty((c,), dtype=torch.float32, device=dev)
    mask = mask if mask is not None else torch.empty((c,), dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = torch.empty((percentile_workspace_bytes(rows, c),), dtype=torch.uint8, device=dev)
    st = lib().hif4_percentile_mask(_ptr(x), rows, c, x.stride(0), float(q), int(n_protect),
                                    _ptr(stats), _ptr(mask), _ptr(workspace), workspace.numel(),
                                    _stream(stream))
    _ok(st, "hif4_percentile_mask")
    return stats, mask


def _check_f32_rows(x, name):
    if x.dtype != torch.float32 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D fp32 CUDA tensor with unit column stride")


def quantize_offsets(x, koff, moff, codes=None, meta=None, stream=None):
    """HiF4-quantize bf16 x [rows][k] with given HiAutoRound offsets: koff fp32
    [rows][k/4] (level-3 exponents), moff fp32 [rows][k] (mantissas).
    Returns (codes u8, meta int32)."""
    _check_bf16_rows(x, "x")
    rows, k = x.shape
    for t, name, shape in ((koff, "koff", (rows, k // 4)), (moff, "moff", (rows, k))):
        if (t.dtype != torch.float32 or not t.is_cuda or tuple(t.shape) != shape
                or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor of shape {shape}")
    dev = x.device
    codes = codes if codes is not None else torch.empty((rows, k // 2), dtype=torch.uint8, device=dev)
    meta = meta if meta is not None else torch.empty((rows, k // 64), dtype=torch.int32, device=dev)
    st = lib().hif4_quantize_offsets(_ptr(x), rows, k, x.stride(0), _ptr(koff), _ptr(moff),
                                     _ptr(codes), _ptr(meta), _stream(stream))
    _ok(st, "hif4_quantize_offsets")
    return codes, meta


def quantize_f32(x, codes=None, meta=None, stream=None):
    """HiF4-quantize fp32 x [rows][k] along k -> (codes u8, meta int32)."""
    _check_f32_rows(x, "x")
    rows, k = x.shape
    dev = x.device
    codes = codes if codes is not None else torch.empty((rows, k // 2), dtype=torch.uint8, device=dev)
    meta = meta if meta is not None else torch.empty((rows, k // 64), dtype=torch.int32, device=dev)
    st = lib().hif4_quantize_f32(_ptr(x), rows, k, x.stride(0), _ptr(codes), _ptr(meta),
                                 _stream(stream))
    _ok(st, "hif4_quantize_f32")
    return codes, meta


def higptq_workspace_bytes(n):
    return int(lib().hif4_higptq_workspace_bytes(n))


def higptq_unit(w, u, unit, codes, meta, workspace=None, stream=None, scheme=1):
    """One HiGPTQ group step (scheme 1, 2 or 3) in place on the fp32 working
    weights w [n][k] with the upper factor u [k][k] (H^-1 = u^T u): writes
    unit ``unit`` of codes/meta and updates the later columns of w."""
    _check_f32_rows(w, "w")
    _check_f32_rows(u, "u")
    n, k = w.shape
    if workspace is None:
        workspace = torch.empty((higptq_workspace_bytes(n),), dtype=torch.uint8, device=w.device)
    st = lib().hif4_higptq_unit(_ptr(w), n, k, w.stride(0), _ptr(u), u.stride(0), int(unit),
                                int(scheme), _ptr(codes), _ptr(meta), _ptr(workspace),
                                workspace.numel(), _stream(stream))
    _ok(st, "hif4_higptq_unit")


HIGPTQ_MAX_BLOCK_UNITS = 16


def higptq_block_workspace_bytes(n, units):
    return int(lib().hif4_higptq_block_workspace_bytes(n, units))


def higptq_block(w, u, unit0, units, codes, meta, workspace=None, stream=None, scheme=1):
    """One HiGPTQ block step (blocksize 64 * units columns, groups unit0 ..
    unit0 + units - 1, scheme 1, 2 or 3) in place on the fp32 working weights
    w [n][k]: writes those units of codes/meta and updates the later columns
    of w, the block's own later columns after each group and the columns after
    the block once."""
    _check_f32_rows(w, "w")
    _check_f32_rows(u, "u")
    n, k = w.shape
    if workspace is None:
        nbytes = max(higptq_block_workspace_bytes(n, units), 1)
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=w.device)
    st = lib().hif4_higptq_block(_ptr(w), n, k, w.stride(0), _ptr(u), u.stride(0), int(unit0),
                                 int(units), int(scheme), _ptr(codes), _ptr(meta),
                                 _ptr(workspace), workspace.numel(), _stream(stream))
    _ok(st, "hif4_higptq_block")


def higptq(w, u, stream=None, scheme=1, block_units=8):
    """HiGPTQ over all groups in blocks of ``block_units`` groups (1 = one
    group at a time through hif4_higptq_unit): returns (codes, meta); w is
    updated in place (its final contents are the compensated working
    weights)."""
    n, k = w.shape
    units = k // 64
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    meta = torch.empty((n, units), dtype=torch.int32, device=w.device)
    if block_units == 1:
        ws = torch.empty((higptq_workspace_bytes(n),), dtype=torch.uint8, device=w.device)
        for unit in range(units):
            higptq_unit(w, u, unit, codes, meta, workspace=ws, stream=stream, scheme=scheme)
        return codes, meta
    ws = torch.empty((max(higptq_block_workspace_bytes(n, block_units), 1),), dtype=torch.uint8,
                     device=w.device)
    for unit0 in range(0, units, block_units):
        higptq_block(w, u, unit0, min(block_units, units - unit0), codes, meta, workspace=ws,
                     stream=stream, scheme=scheme)
    return codes, meta


# ---------------------------------------------------------------- 8-bit linear layers
#
# Codes are torch.float8_e4m3fn, power-of-two scales torch.float8_e8m0fnu (a
# view of rows padded to whole 32-bit words: the stride is a multiple of 4).

FP8_BLOCK = 128
HIF4_SCALE_E8M0, HIF4_SCALE_F32 = 0, 1
_DTYPE = {torch.float32: HIF4_F32, torch.bfloat16: HIF4_BF16}


class _On:
    """The device of a call's tensors and the stream its work goes to: checks
    that every tensor given is on that device, makes it current, and allocates
    outputs and workspaces on that stream (so their memory is not handed out
    again while the stream still uses it). Switches nothing where the current
    device and stream are the call's."""

    __slots__ = ("_ctx", "_raw")

    def __init__(self, first, stream, *tensors):
        if not first.is_cuda:
            raise ValueError("tensors must be on the GPU")
        index = first.get_device()
        for t in tensors:
            if t is not None and t.get_device() != index:
                raise ValueError(f"a tensor is on {t.device}, the call's first one on {first.device}")
        self._ctx = None
        if stream is not None:
            if stream.device_index != index:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {first.device}")
            self._raw = stream.cuda_stream
            self._ctx = torch.cuda.stream(stream)  # makes the stream's device current, too
        else:
            self._raw = torch._C._cuda_getCurrentRawStream(index)
            if torch._C._cuda_getDevice() != index:
                self._ctx = torch.cuda.device(index)

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        return self._raw

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        return False


def _at(t):
    """Address of a tensor, or None."""
    return t.data_ptr() if t is not None else None


def _check_rows(x, name):
    if x.dtype not in _DTYPE or x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D fp32 or bf16 tensor with unit column stride")


def _ld(t):
    """Leading dimension of a 2-D tensor (a single row's stride says nothing)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _up128(v):
    return (v + 127) // 128 * 128


def _empty_scales(rows, blocks, device):
    full = torch.empty((rows, (blocks + 3) // 4 * 4), dtype=torch.float8_e8m0fnu, device=device)
    return full if blocks % 4 == 0 else full[:, :blocks]


def _check_out(t, name, shape, dtype):
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {shape}")


def _workspace_bytes(t):
    if not t.is_contiguous():  # its elements may share memory
        raise ValueError("workspace must be contiguous")
    return t.numel() * t.element_size()


def _check_scales(t, name, rows, blocks):
    """E8M0 scales [rows][blocks] whose rows are whole 32-bit words in memory."""
    if t.dtype != torch.float8_e8m0fnu or tuple(t.shape) != (rows, blocks):
        raise ValueError(f"{name} must be a float8_e8m0fnu tensor of shape {(rows, blocks)}")
    if rows == 0 or blocks == 0:
        return
    ld = _ld(t)
    held = t.untyped_storage().nbytes() - t.storage_offset()
    if (blocks > 1 and t.stride(1) != 1) or ld % 4 or ld < blocks or held < (rows - 1) * ld + (blocks + 3) // 4 * 4:
        raise ValueError(f"{name}: rows must be padded to a multiple of 4 bytes (stride {ld} for "
                         f"{blocks} blocks)")


def _scale_ld(t):
    blocks = t.shape[1]
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), (blocks + 3) // 4 * 4)


def _fp8_out(rows, length, block_rows, codes, scales, dev):
    """Codes [rows][length up to 128s] and their scales, given or new."""
    cols = _up128(length)
    srows = (rows + block_rows - 1) // block_rows
    if codes is None:
        codes = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=dev)
    else:
        _check_out(codes, "codes", (rows, cols), torch.float8_e4m3fn)
    if scales is None:
        scales = _empty_scales(srows, cols // FP8_BLOCK, dev)
    else:
        _check_scales(scales, "scales", srows, cols // FP8_BLOCK)
    return codes, scales


def _check_block_rows(block_rows):
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError("block_rows must be 1 or 128")


def quantize_fp8(x, block_rows=1, transposed=False, codes=None, scales=None, stream=None):
    """E4M3-quantize x [rows][k] (bf16 or fp32) in blocks of 128 along k, or with
    transposed=True x^T in blocks along the rows of x; block_rows=128: 128 x 128
    tiles. Returns (codes [rows][k up to 128s], scales [rows / block_rows][blocks])."""
    _check_rows(x, "x")
    _check_block_rows(block_rows)
    rows, k = x.shape
    with _On(x, stream, codes, scales) as st:
        out = (k, rows) if transposed else (rows, k)
        codes, scales = _fp8_out(*out, block_rows, codes, scales, x.device)
        _ok(lib().hif4_quantize_fp8(_at(x), _DTYPE[x.dtype], rows, k, _ld(x), block_rows,
                                    int(bool(transposed)), _at(codes), _at(scales),
                                    _scale_ld(scales), st), "hif4_quantize_fp8")
    return codes, scales


def quantize_fp8_both(x, block_rows=1, stream=None):
    """quantize_fp8 of x and of x^T from one read: (codes, scales, codes_t, scales_t)."""
    _check_rows(x, "x")
    _check_block_rows(block_rows)
    rows, k = x.shape
    with _On(x, stream) as st:
        codes, scales = _fp8_out(rows, k, block_rows, None, None, x.device)
        codes_t, scales_t = _fp8_out(k, rows, block_rows, None, None, x.device)
        _ok(lib().hif4_quantize_fp8_both(_at(x), _DTYPE[x.dtype], rows, k, _ld(x), block_rows,
                                         _at(codes), _at(scales), _scale_ld(scales),
                                         _at(codes_t), _at(scales_t), _scale_ld(scales_t), st),
            "hif4_quantize_fp8_both")
    return codes, scales, codes_t, scales_t


def _check_codes(codes, name):
    if (codes.dtype != torch.float8_e4m3fn or codes.dim() != 2 or not codes.is_contiguous()
            or codes.shape[1] % FP8_BLOCK):
        raise ValueError(f"{name} must be a contiguous 2-D float8_e4m3fn tensor, its rows a multiple "
                         "of 128 long")


def _weight_scales(scales, n, blocks, name):
    """(scale type, block_rows, leading dimension) of a weight's scales."""
    tiles = (n + FP8_BLOCK - 1) // FP8_BLOCK
    if scales.dtype == torch.float32:
        if tuple(scales.shape) != (tiles, blocks) or (blocks > 1 and scales.stride(1) != 1):
            raise ValueError(f"{name}: float32 scales are one per 128 x 128 tile, {(tiles, blocks)}, "
                             "with unit column stride")
        return HIF4_SCALE_F32, FP8_BLOCK, _ld(scales)
    rows = scales.shape[0] if scales.dim() == 2 and scales.shape[0] in (n, tiles) else n
    _check_scales(scales, name, rows, blocks)
    return HIF4_SCALE_E8M0, (1 if rows == n else FP8_BLOCK), _scale_ld(scales)


def dequantize_fp8(codes, scales, k=None, out_dtype=torch.float32, out=None, stream=None):
    """Values [rows][k] (fp32 or bf16) of codes and scales (E8M0 per 1 x 128 or
    128 x 128, or float32 per 128 x 128); k: the columns before the padding."""
    _check_codes(codes, "codes")
    rows, kp = codes.shape
    k = kp if k is None else int(k)
    if _up128(k) != kp or k < 0:
        raise ValueError(f"k = {k} does not fit codes of {kp} columns")
    if out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    with _On(codes, stream, scales, out) as st:
        kind, block_rows, ld = _weight_scales(scales, rows, kp // FP8_BLOCK, "scales")
        if out is None:
            out = torch.empty((rows, k), dtype=out_dtype, device=codes.device)
        else:
            _check_out(out, "out", (rows, k), out_dtype)
        _ok(lib().hif4_dequantize_fp8(_at(codes), _at(scales), kind, block_rows, ld, rows, k,
                                      _at(out), _DTYPE[out_dtype], st), "hif4_dequantize_fp8")
    return out


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def linear_fp8_workspace_bytes(m, n, k):
    return int(lib().hif4_linear_fp8_workspace_bytes(m, n, k))


def linear_fp8(x_codes, x_scales, w_codes, w_scales, y_dtype=torch.float32, y=None, workspace=None,
               stream=None):
    """Y [m][n] = X W^T of E4M3 codes x_codes [m][k] (E8M0 scales per 1 x 128) and
    w_codes [n][k] (E8M0 scales per 1 x 128 or 128 x 128, or float32 per 128 x 128).

    A float32 Y is a full fp32 sum of exact products (for scale bytes 3 to 246; the
    header states the rest). A bfloat16 Y comes from the fp8 matrix instructions, which
    cut each product to 2^-13 of the largest of its run of 8 along k: at most
    7 * 2^-13 of sum |x||w| is lost, on random signs some 1e-5 of |Y|, but all of the
    small products beside large ones that cancel. Take float32 where those count. Up to
    16 rows either type is the full sum."""
    _check_codes(x_codes, "x_codes")
    _check_codes(w_codes, "w_codes")
    (m, k), n = x_codes.shape, w_codes.shape[0]
    if w_codes.shape[1] != k:
        raise ValueError(f"x_codes has {k} columns, w_codes {w_codes.shape[1]}")
    if y_dtype not in _DTYPE:
        raise ValueError("y_dtype must be float32 or bfloat16")
    with _On(x_codes, stream, x_scales, w_codes, w_scales, y, workspace) as st:
        _check_scales(x_scales, "x_scales", m, k // FP8_BLOCK)
        kind, block_rows, ldws = _weight_scales(w_scales, n, k // FP8_BLOCK, "w_scales")
        if y is None:
            y = torch.empty((m, n), dtype=y_dtype, device=x_codes.device)
        else:
            _check_out(y, "y", (m, n), y_dtype)
        need = linear_fp8_workspace_bytes(m, n, k)
        if workspace is None and need:
            workspace = torch.empty((need,), dtype=torch.uint8, device=x_codes.device)
        nbytes = _workspace_bytes(workspace) if workspace is not None else 0
        _ok(lib().hif4_linear_fp8(_at(x_codes), _at(x_scales), _scale_ld(x_scales), _at(w_codes),
                                  _at(w_scales), ldws, kind, block_rows, m, n, k, _at(y),
                                  _DTYPE[y_dtype], _at(workspace), nbytes, st), "hif4_linear_fp8")
    return y


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def linear_fp8_backward_workspace_bytes(m, n, k):
    return int(lib().hif4_linear_fp8_backward_workspace_bytes(m, n, k))


def linear_fp8_backward(dy, xt_codes, xt_scales, wt_codes, wt_scales, dx_dtype=None,
                        dw_dtype=torch.float32, workspace=None, stream=None):
    """Gradients of Y = X W^T through the quantizers (taken as the identity):
    dX [m][k] = Q(dY) W and dW [n][k] = Q(dY^T) X for dy [m][n] (bf16 or fp32),
    with X^T and W^T quantized along m and n (quantize_fp8(..., transposed=True);
    the weight's scales as linear_fp8 takes them). dX is of dy's type unless
    dx_dtype says otherwise. Each gradient has linear_fp8's precision for its type: a
    bfloat16 dX, the default for a bfloat16 dy, is cut as a bfloat16 Y is (to at most
    7 * 2^-13 of sum |dy||w|); dx_dtype=torch.float32 gives the full fp32 sum, as dw's
    default does."""
    _check_rows(dy, "dy")
    _check_codes(xt_codes, "xt_codes")
    _check_codes(wt_codes, "wt_codes")
    (m, n), k = dy.shape, xt_codes.shape[0]
    mp, np_ = _up128(m), _up128(n)
    if xt_codes.shape[1] != mp or wt_codes.shape != (k, np_):
        raise ValueError(f"dy is {m} x {n}: xt_codes must be [k][{mp}], wt_codes [k][{np_}]")
    dx_dtype = dy.dtype if dx_dtype is None else dx_dtype
    if dx_dtype not in _DTYPE or dw_dtype not in _DTYPE:
        raise ValueError("dx_dtype and dw_dtype must be float32 or bfloat16")
    with _On(dy, stream, xt_codes, xt_scales, wt_codes, wt_scales, workspace) as st:
        _check_scales(xt_scales, "xt_scales", k, mp // FP8_BLOCK)
        kind, block_rows, ldwt = _weight_scales(wt_scales, k, np_ // FP8_BLOCK, "wt_scales")
        dx = torch.empty((m, k), dtype=dx_dtype, device=dy.device)
        dw = torch.empty((n, k), dtype=dw_dtype, device=dy.device)
        if workspace is None:
            workspace = torch.empty((linear_fp8_backward_workspace_bytes(m, n, k),),
                                    dtype=torch.uint8, device=dy.device)
        _ok(lib().hif4_linear_fp8_backward(_at(dy), _DTYPE[dy.dtype], _ld(dy), _at(xt_codes),
                                           _at(xt_scales), _scale_ld(xt_scales), _at(wt_codes),
                                           _at(wt_scales), ldwt, kind, block_rows, m, n, k, _at(dx),
                                           _DTYPE[dx_dtype], _at(dw), _DTYPE[dw_dtype],
                                           _at(workspace),
                                           _workspace_bytes(workspace), st),
            "hif4_linear_fp8_backward")
    return dx, dw


# ---------------------------------------------------------------- 4-bit microscaled linear layers
#
# A matrix [rows][k] is codes uint8 [rows][kp/2] and scales torch.float8_e8m0fnu
# [rows][kp/32], kp = k up to 128s, both contiguous; experts' weights have one more
# dimension in front. Groups of rows are an int64 tensor of offsets on the GPU: group e
# is rows offsets[e] .. offsets[e + 1] - 1.

MXFP4_BLOCK = 32


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def mxfp4_columns(rows, groups=0):
    """Columns of a transpose quantized along its source's rows (in `groups` groups)."""
    return int(lib().hif4_mxfp4_columns(rows, groups))


def _check_offsets(offsets):
    """Number of groups of an offsets tensor."""
    if offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() < 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int64 tensor [groups + 1]")
    return offsets.numel() - 1


_U8, _E8 = torch.uint8, torch.float8_e8m0fnu


def _mx4_out(like, lead, rows, length, codes, scales):
    """Codes [*lead, rows, length up to 128s / 2] and their scales, given or new beside `like`."""
    kp = _up128(length)
    if codes is None:
        codes = like.new_empty((*lead, rows, kp // 2), dtype=_U8)
    else:
        _check_out(codes, "codes", (*lead, rows, kp // 2), _U8)
    if scales is None:
        scales = like.new_empty((*lead, rows, kp // MXFP4_BLOCK), dtype=_E8)
    else:
        _check_out(scales, "scales", (*lead, rows, kp // MXFP4_BLOCK), _E8)
    return codes, scales


def _mx4_x(x, offsets, transposed):
    """(batch, rows, k, ld, leading dimensions, groups) of what is quantized."""
    if x.dim() == 3:
        if x.dtype not in _DTYPE or not x.is_contiguous():
            raise ValueError("x must be a contiguous fp32 or bf16 tensor where it has three dimensions")
        batch, rows, k = x.shape
        ld, lead = k, (batch,)
    else:
        _check_rows(x, "x")
        (rows, k), batch, ld, lead = x.shape, 1, _ld(x), ()
    if offsets is None:
        return batch, rows, k, ld, lead, 0
    groups = _check_offsets(offsets)
    if not transposed or lead or groups == 0:
        raise ValueError("offsets (of one group at least) go with a 2-D x quantized along its rows")
    return batch, rows, k, ld, lead, groups


def quantize_mxfp4(x, transposed=False, offsets=None, codes=None, scales=None, stream=None):
    """MXFP4-quantize x [rows][k] (bf16 or fp32; or [experts][rows][k]) in blocks of 32
    along k, or with transposed=True x^T in blocks along the rows of x, with `offsets`
    each group's rows by themselves. Returns (codes [rows][k up to 128s / 2], scales
    [rows][k up to 128s / 32]), or those of x^T, whose columns are
    mxfp4_columns(rows, groups)."""
    batch, rows, k, ld, lead, groups = _mx4_x(x, offsets, transposed)
    with _On(x, stream, offsets, codes, scales) as st:
        out = (k, mxfp4_columns(rows, groups)) if transposed else (rows, k)
        codes, scales = _mx4_out(x, lead, *out, codes, scales)
        _ok(lib().hif4_quantize_mxfp4(_at(x), _DTYPE[x.dtype], batch, rows, k, ld, int(bool(transposed)),
                                      _at(offsets), groups, _at(codes), _at(scales), st),
            "hif4_quantize_mxfp4")
    return codes, scales


def quantize_mxfp4_both(x, offsets=None, stream=None):
    """quantize_mxfp4 of x and of x^T (in groups of its rows) from one read: (codes,
    scales, codes_t, scales_t). Codes and scales of rows outside every group are not
    written."""
    batch, rows, k, ld, lead, groups = _mx4_x(x, offsets, True)
    with _On(x, stream, offsets) as st:
        codes, scales = _mx4_out(x, lead, rows, k, None, None)
        codes_t, scales_t = _mx4_out(x, lead, k, mxfp4_columns(rows, groups), None, None)
        _ok(lib().hif4_quantize_mxfp4_both(_at(x), _DTYPE[x.dtype], batch, rows, k, ld, _at(offsets), groups,
                                           _at(codes), _at(scales), _at(codes_t), _at(scales_t), st),
            "hif4_quantize_mxfp4_both")
    return codes, scales, codes_t, scales_t


def _check_mx4(codes, scales, name, dims=2):
    """Codes [..., rows, kp/2] with scales [..., rows, kp/32]: their leading sizes and kp."""
    *lead, half = codes.shape
    *lead_s, blocks = scales.shape
    if (codes.dtype is _U8 and scales.dtype is _E8 and half == 16 * blocks and half % 64 == 0
            and lead == lead_s and len(lead) == dims - 1 and codes.is_contiguous() and scales.is_contiguous()):
        return *lead, 2 * half
    raise ValueError(f"{name}_codes must be a contiguous {dims}-D uint8 tensor, its rows a multiple of 64 bytes (128 "
                     f"codes) long, and {name}_scales a contiguous float8_e8m0fnu tensor of the same rows, a byte for "
                     f"each 16 of codes; they are {codes.dtype} {tuple(codes.shape)} and {scales.dtype} "
                     f"{tuple(scales.shape)}")


def dequantize_mxfp4(codes, scales, k=None, out_dtype=torch.float32, out=None, stream=None):
    """Values [rows][k] (fp32 or bf16; [experts][rows][k] of such codes) of codes and
    scales; k: the columns before the padding."""
    *lead, kp = _check_mx4(codes, scales, "mxfp4", codes.dim() if codes.dim() in (2, 3) else 2)
    k = kp if k is None else int(k)
    if _up128(k) != kp or k < 0:
        raise ValueError(f"k = {k} does not fit codes of {kp} columns")
    if out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    with _On(codes, stream, scales, out) as st:
        if out is None:
            out = codes.new_empty((*lead, k), dtype=out_dtype)
        else:
            _check_out(out, "out", (*lead, k), out_dtype)
        rows = lead[0] if len(lead) == 1 else lead[0] * lead[1]
        _ok(lib().hif4_dequantize_mxfp4(_at(codes), _at(scales), rows, k, _at(out), _DTYPE[out_dtype], st),
            "hif4_dequantize_mxfp4")
    return out


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def linear_mxfp4_workspace_bytes(m, n, k):
    return int(lib().hif4_linear_mxfp4_workspace_bytes(m, n, k))


def _y_out(like, y, m, n, y_dtype):
    if y_dtype not in _DTYPE:
        raise ValueError("y_dtype must be float32 or bfloat16")
    if y is None:
        return like.new_empty((m, n), dtype=y_dtype)
    _check_out(y, "y", (m, n), y_dtype)
    return y


def linear_mxfp4(x_codes, x_scales, w_codes, w_scales, y_dtype=torch.float32, y=None, workspace=None,
                 stream=None):
    """Y [m][n] = X W^T of MXFP4 X [m][k] and W [n][k]: exact products, fp32 sums,
    rounded once."""
    m, k = _check_mx4(x_codes, x_scales, "x")
    n, kw = _check_mx4(w_codes, w_scales, "w")
    if kw != k:
        raise ValueError(f"x has {k} columns, w {kw}")
    with _On(x_codes, stream, x_scales, w_codes, w_scales, y, workspace) as st:
        y = _y_out(x_codes, y, m, n, y_dtype)
        need = linear_mxfp4_workspace_bytes(m, n, k)
        if workspace is None and need:
            workspace = torch.empty((need,), dtype=torch.uint8, device=x_codes.device)
        nbytes = _workspace_bytes(workspace) if workspace is not None else 0
        _ok(lib().hif4_linear_mxfp4(_at(x_codes), _at(x_scales), _at(w_codes), _at(w_scales), m, n, k,
                                    _at(y), _DTYPE[y_dtype], _at(workspace), nbytes, st),
            "hif4_linear_mxfp4")
    return y


def linear_mxfp4_grouped(x_codes, x_scales, w_codes, w_scales, offsets, y_dtype=torch.float32, y=None,
                         stream=None):
    """Y [m][n]: Y[i] = X[i] W[e]^T for the rows i of each group e (rows offsets[e] ..
    offsets[e + 1] - 1), MXFP4 X [m][k] and W [experts][n][k]. Rows outside every group
    are not written."""
    m, k = _check_mx4(x_codes, x_scales, "x")
    experts, n, kw = _check_mx4(w_codes, w_scales, "w", 3)
    groups = _check_offsets(offsets)
    if kw != k or experts != groups:
        raise ValueError(f"x has {k} columns and offsets {groups} groups, w {kw} columns and {experts} experts")
    with _On(x_codes, stream, x_scales, w_codes, w_scales, offsets, y) as st:
        y = _y_out(x_codes, y, m, n, y_dtype)
        _ok(lib().hif4_linear_mxfp4_grouped(_at(x_codes), _at(x_scales), _at(w_codes), _at(w_scales),
                                            _at(offsets), groups, m, n, k, _at(y), _DTYPE[y_dtype], st),
            "hif4_linear_mxfp4_grouped")
    return y


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def linear_mxfp4_backward_workspace_bytes(m, n, k):
    return int(lib().hif4_linear_mxfp4_backward_workspace_bytes(m, n, k))


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def linear_mxfp4_grouped_backward_workspace_bytes(groups, m, n, k):
    return int(lib().hif4_linear_mxfp4_grouped_backward_workspace_bytes(groups, m, n, k))


def _mx4_gradient_types(dy, dx_dtype, dw_dtype):
    dx_dtype = dy.dtype if dx_dtype is None else dx_dtype
    if dx_dtype not in _DTYPE or dw_dtype not in _DTYPE:
        raise ValueError("dx_dtype and dw_dtype must be float32 or bfloat16")
    return dx_dtype


def linear_mxfp4_backward(dy, xt_codes, xt_scales, wt_codes, wt_scales, dx_dtype=None,
                          dw_dtype=torch.float32, workspace=None, stream=None, need_dx=True, need_dw=True):
    """Gradients of Y = X W^T through the quantizers (taken as the identity): dX [m][k] =
    Q(dY) W and dW [n][k] = Q(dY^T) X for dy [m][n] (bf16 or fp32), with X^T and W^T
    quantized along m and n (quantize_mxfp4(..., transposed=True)). dX is of dy's type
    unless dx_dtype says otherwise. A gradient that is not needed is None and costs
    nothing; without dX wt_codes and wt_scales may be None, without dW xt_codes and
    xt_scales."""
    _check_rows(dy, "dy")
    if not (need_dx or need_dw):
        raise ValueError("one of need_dx and need_dw has to be set")
    m, n = dy.shape
    k = mp = np_ = None
    if need_dw:
        k, mp = _check_mx4(xt_codes, xt_scales, "xt")
    if need_dx:
        kw, np_ = _check_mx4(wt_codes, wt_scales, "wt")
        k = kw if k is None else k
    if (need_dx and (kw != k or np_ != _up128(n))) or (need_dw and mp != _up128(m)):
        raise ValueError(f"dy is {m} x {n}: xt must be [k][{_up128(m)}], wt [k][{_up128(n)}]")
    dx_dtype = _mx4_gradient_types(dy, dx_dtype, dw_dtype)
    xt = (xt_codes, xt_scales) if need_dw else (None, None)
    wt = (wt_codes, wt_scales) if need_dx else (None, None)
    with _On(dy, stream, *xt, *wt, workspace) as st:
        dx = dy.new_empty((m, k), dtype=dx_dtype) if need_dx else None
        dw = dy.new_empty((n, k), dtype=dw_dtype) if need_dw else None
        if workspace is None:
            workspace = dy.new_empty((linear_mxfp4_backward_workspace_bytes(m, n, k),), dtype=_U8)
        _ok(lib().hif4_linear_mxfp4_backward(_at(dy), _DTYPE[dy.dtype], _ld(dy), _at(xt[0]), _at(xt[1]),
                                             _at(wt[0]), _at(wt[1]), m, n, k, _at(dx), _DTYPE[dx_dtype],
                                             _at(dw), _DTYPE[dw_dtype], _at(workspace),
                                             _workspace_bytes(workspace), st),
            "hif4_linear_mxfp4_backward")
    return dx, dw


def linear_mxfp4_grouped_backward(dy, xt_codes, xt_scales, wt_codes, wt_scales, offsets, dx_dtype=None,
                                  dw_dtype=torch.float32, workspace=None, stream=None, need_dx=True,
                                  need_dw=True):
    """Gradients of linear_mxfp4_grouped: dX [m][k], dX[i] = Q(dY)[i] W[e] for the rows i
    of each group e, and dW [experts][n][k], dW[e] = Q(dY_e^T) X_e (0 for a group without
    rows), for dy [m][n], with X^T quantized along each group's rows
    (quantize_mxfp4(x, transposed=True, offsets=offsets)) and the experts' W^T along n
    (quantize_mxfp4(w, transposed=True)). Rows of dX outside every group are not
    written. need_dx and need_dw as for linear_mxfp4_backward."""
    _check_rows(dy, "dy")
    if not (need_dx or need_dw):
        raise ValueError("one of need_dx and need_dw has to be set")
    m, n = dy.shape
    groups = _check_offsets(offsets)
    want = mxfp4_columns(m, groups) if groups else 0
    k = mp = None
    if need_dw:
        k, mp = _check_mx4(xt_codes, xt_scales, "xt")
    if need_dx:
        experts, kw, np_ = _check_mx4(wt_codes, wt_scales, "wt", 3)
        k = kw if k is None else k
    if (need_dx and (kw != k or experts != groups or np_ != _up128(n))) or (need_dw and mp != want):
        raise ValueError(f"dy is {m} x {n} in {groups} groups: xt must be [k][{want}], wt [{groups}][k]"
                         f"[{_up128(n)}]")
    dx_dtype = _mx4_gradient_types(dy, dx_dtype, dw_dtype)
    xt = (xt_codes, xt_scales) if need_dw else (None, None)
    wt = (wt_codes, wt_scales) if need_dx else (None, None)
    with _On(dy, stream, *xt, *wt, offsets, workspace) as st:
        dx = dy.new_empty((m, k), dtype=dx_dtype) if need_dx else None
        dw = dy.new_empty((groups, n, k), dtype=dw_dtype) if need_dw else None
        if workspace is None:
            need = linear_mxfp4_grouped_backward_workspace_bytes(groups, m, n, k)
            workspace = dy.new_empty((need,), dtype=_U8)
        _ok(lib().hif4_linear_mxfp4_grouped_backward(_at(dy), _DTYPE[dy.dtype], _ld(dy), _at(xt[0]), _at(xt[1]),
                                                     _at(wt[0]), _at(wt[1]), _at(offsets), groups, m, n, k,
                                                     _at(dx), _DTYPE[dx_dtype], _at(dw), _DTYPE[dw_dtype],
                                                     _at(workspace), _workspace_bytes(workspace), st),
            "hif4_linear_mxfp4_grouped_backward")
    return dx, dw


# ---------------------------------------------------------------- layer norm


def _check_affine(weight, bias, c):
    """(weight, bias) dtype code; float32 when neither is given."""
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None and (t.dtype not in _DTYPE or tuple(t.shape) != (c,) or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous fp32 or bf16 tensor of shape {(c,)}")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one dtype")
    first = weight if weight is not None else bias
    return HIF4_F32 if first is None else _DTYPE[first.dtype]


def layer_norm(x, weight=None, bias=None, eps=1e-6, y=None, stream=None):
    """Layer norm over the rows of x [rows][c] (bf16 or fp32): (y, mean, rstd), y
    of x's dtype, mean and rstd float32 [rows] for the backward."""
    _check_rows(x, "x")
    rows, c = x.shape
    wd = _check_affine(weight, bias, c)
    with _On(x, stream, weight, bias, y) as st:
        if y is None:
            y = x.new_empty((rows, c))
        elif y.dtype != x.dtype or y.shape != x.shape or (c > 1 and y.stride(1) != 1):
            raise ValueError("y must have x's dtype and shape and unit column stride")
        mean = x.new_empty((rows,), dtype=torch.float32)
        rstd = torch.empty_like(mean)
        _ok(lib().hif4_layer_norm(_at(x), _DTYPE[x.dtype], rows, c, _ld(x), _at(weight),
                                  _at(bias), wd, float(eps), _at(y), _ld(y), _at(mean),
                                  _at(rstd), st), "hif4_layer_norm")
    return y, mean, rstd


def layer_norm_quantize(x, weight=None, bias=None, eps=1e-6, mask=None, codes=None, meta=None,
                        stream=None):
    """layer_norm (rounded to bf16) and quantize in one pass: (codes, meta, kept),
    what linear_w4a4 takes as x_codes, x_meta and x_kept."""
    _check_rows(x, "x")
    rows, c = x.shape
    wd = _check_affine(weight, bias, c)
    if c % 64:
        raise ValueError(f"HiF4 units are 64 wide: {c} columns")
    with _On(x, stream, weight, bias, mask, codes, meta) as st:
        n_mask, kept = 0, None
        if mask is not None:
            if mask.dtype != torch.uint8 or tuple(mask.shape) != (c,) or not mask.is_contiguous():
                raise ValueError(f"mask must be a contiguous uint8 tensor of shape {(c,)}")
            n_mask = int(torch.count_nonzero(mask).item())
            kept = torch.empty((rows, n_mask), dtype=torch.bfloat16, device=x.device)
        if codes is None:
            codes = torch.empty((rows, c // 2), dtype=torch.uint8, device=x.device)
        else:
            _check_out(codes, "codes", (rows, c // 2), torch.uint8)
        if meta is None:
            meta = torch.empty((rows, c // 64), dtype=torch.int32, device=x.device)
        else:
            _check_out(meta, "meta", (rows, c // 64), torch.int32)
        _ok(lib().hif4_layer_norm_quantize(_at(x), _DTYPE[x.dtype], rows, c, _ld(x), _at(weight),
                                           _at(bias), wd, float(eps), _at(mask), n_mask,
                                           _at(kept) if n_mask else None, _at(codes), _at(meta),
                                           st), "hif4_layer_norm_quantize")
    return codes, meta, kept


def layer_norm_quantize_fp8(x, weight=None, bias=None, eps=1e-6, codes=None, scales=None,
                            stream=None):
    """layer_norm and quantize_fp8 (blocks of 1 x 128) in one pass: (codes, scales),
    what linear_fp8 takes as x_codes and x_scales."""
    _check_rows(x, "x")
    rows, c = x.shape
    wd = _check_affine(weight, bias, c)
    with _On(x, stream, weight, bias, codes, scales) as st:
        codes, scales = _fp8_out(rows, c, 1, codes, scales, x.device)
        _ok(lib().hif4_layer_norm_quantize_fp8(_at(x), _DTYPE[x.dtype], rows, c, _ld(x),
                                               _at(weight), _at(bias), wd, float(eps),
                                               _at(codes), _at(scales), _scale_ld(scales), st),
            "hif4_layer_norm_quantize_fp8")
    return codes, scales


def layer_norm_quantize_mxfp4(x, weight=None, bias=None, eps=1e-6, codes=None, scales=None, stream=None):
    """layer_norm and quantize_mxfp4 in one pass: (codes, scales), what linear_mxfp4 takes
    as x_codes and x_scales."""
    _check_rows(x, "x")
    rows, c = x.shape
    wd = _check_affine(weight, bias, c)
    with _On(x, stream, weight, bias, codes, scales) as st:
        codes, scales = _mx4_out(x, (), rows, c, codes, scales)
        _ok(lib().hif4_layer_norm_quantize_mxfp4(_at(x), _DTYPE[x.dtype], rows, c, _ld(x), _at(weight),
                                                 _at(bias), wd, float(eps), _at(codes), _at(scales), st),
            "hif4_layer_norm_quantize_mxfp4")
    return codes, scales


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def layer_norm_backward_workspace_bytes(rows, c):
    return int(lib().hif4_layer_norm_backward_workspace_bytes(rows, c))


def layer_norm_backward(dy, x, mean, rstd, weight=None, workspace=None, stream=None):
    """Gradients of layer_norm: (dx, dweight, dbias); dweight and dbias in the
    weight's dtype (float32 without a weight)."""
    _check_rows(x, "x")
    _check_rows(dy, "dy")
    rows, c = x.shape
    if dy.dtype != x.dtype or dy.shape != x.shape:
        raise ValueError("dy must have x's dtype and shape")
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != torch.float32 or tuple(t.shape) != (rows,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {(rows,)}")
    wd = _check_affine(weight, None, c)
    with _On(x, stream, dy, mean, rstd, weight, workspace) as st:
        dx = x.new_empty((rows, c))
        dweight = torch.empty_like(weight) if weight is not None else mean.new_empty((c,))
        dbias = torch.empty_like(dweight)
        if workspace is None:
            need = max(layer_norm_backward_workspace_bytes(rows, c), 1)
            workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
        _ok(lib().hif4_layer_norm_backward(_at(dy), _ld(dy), _at(x), _ld(x), _DTYPE[x.dtype], rows,
                                           c, _at(mean), _at(rstd), _at(weight), wd, _at(dx), c,
                                           _at(dweight), _at(dbias), _at(workspace),
                                           _workspace_bytes(workspace), st),
            "hif4_layer_norm_backward")
    return dx, dweight, dbias
