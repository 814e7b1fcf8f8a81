"""ctypes binding of libmx.so (the C ABI in include/mx.h).

Argument marshalling only: every step of quantization, dequantization and
the GEMM runs in the HIP kernels of libmx.so.  PyTorch supplies device
memory and the current HIP stream.  If the library is not built, calls raise
immediately; there is no fallback implementation.
"""
import ctypes
import os
from typing import NamedTuple, Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmx.so")

MX_OK, MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED, MX_ERR_ALIGNMENT, MX_ERR_HIP = range(5)
MX_SRC_F32, MX_SRC_BF16 = 0, 1
MX_E4M3, MX_E5M2, MX_E2M1 = 0, 1, 2
MX_SCALE_E8M0, MX_SCALE_E8M0_TENSOR_F32 = 0, 1
MX_TSCALE_COMPUTE, MX_TSCALE_PROVIDED = 0, 1
MX_RNE, MX_SR = 0, 1
MX_AXIS_ROW, MX_AXIS_COL = 0, 1
MX_OUT_F32, MX_OUT_BF16 = 0, 1
MX_NORM_LAYER, MX_NORM_RMS = 0, 1
MX_ACT_SILU, MX_ACT_GELU, MX_ACT_GELU_TANH = 0, 1, 2

FMTS = {"e4m3": MX_E4M3, "e5m2": MX_E5M2, "e2m1": MX_E2M1}
NORMS = {"layer": MX_NORM_LAYER, "rms": MX_NORM_RMS}
ACTS = {"silu": MX_ACT_SILU, "gelu": MX_ACT_GELU, "gelu_tanh": MX_ACT_GELU_TANH}
EXPORTED = ("mx_quantize", "mx_quantize_dual_layout", "mx_gemm", "mx_dequantize",
            "mx_status_string", "mx_last_error_message",
            "mx_predict_tensor_scale", "mx_predict_workspace_bytes", "mx_gemm_quantized",
            "mx_predict_tensor_scale_noalloc", "mx_quantize_optstate", "mx_dequantize_optstate",
            "mx_quantize_nvfp", "mx_dequantize_nvfp", "mx_gemm_nvfp",
            "mx_norm_forward", "mx_norm_backward", "mx_norm_backward_workspace_bytes",
            "mx_glu_forward", "mx_glu_backward", "mx_glu_backward_dual_layout")
NV_PANEL = 32                      # stored rows per CTA-local nvfp scale domain


class MXError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_name(status)}: {message}")
        self.status = status


class mx_qconfig(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("block", ctypes.c_int32),
                ("scale_fmt", ctypes.c_int32), ("tscale", ctypes.c_int32),
                ("rounding", ctypes.c_int32), ("hadamard", ctypes.c_int32),
                ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


_lib = None
_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


def load() -> ctypes.CDLL:
    """Load libmx.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
    L = ctypes.CDLL(LIB_PATH)
    L.mx_quantize.restype = _i32
    L.mx_quantize.argtypes = [_vp, _i32, _i64, _i64, _i64, _i32, ctypes.POINTER(mx_qconfig),
                              _vp, _vp, _vp, _vp]
    L.mx_quantize_dual_layout.restype = _i32
    L.mx_quantize_dual_layout.argtypes = [_vp, _i32, _i64, _i64, _i64,
                                          ctypes.POINTER(mx_qconfig), _vp, _vp, _vp, _vp, _vp,
                                          _vp]
    L.mx_gemm.restype = _i32
    L.mx_gemm.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _i64, _i64, _i64,
                          ctypes.c_float, _i32, _vp, _i32, _i64, _vp]
    L.mx_dequantize.restype = _i32
    L.mx_dequantize.argtypes = [_vp, _vp, _vp, _i32, _i64, _i64, _i32, _i32, _vp, _i32, _vp]
    L.mx_gemm_quantized.restype = _i32
    L.mx_gemm_quantized.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _i64, _i64, _i64,
                                    ctypes.c_float, _i32, _i32, _vp, _vp, _vp]
    L.mx_predict_tensor_scale.restype = _i32
    L.mx_predict_tensor_scale.argtypes = [_vp, _i64, _vp, _i64, _i32, _i64, _i64, ctypes.c_float, _i32,
                                          _vp, _i64, _vp, _vp]
    L.mx_predict_tensor_scale_noalloc.restype = _i32
    L.mx_predict_tensor_scale_noalloc.argtypes = [_vp, _i64, _vp, _i64, _i32, _i64, _i64, ctypes.c_float,
                                                  _i32, _vp, _vp]
    L.mx_quantize_optstate.restype = _i32
    L.mx_quantize_optstate.argtypes = [_vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp]
    L.mx_dequantize_optstate.restype = _i32
    L.mx_dequantize_optstate.argtypes = [_vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp]
    L.mx_quantize_nvfp.restype = _i32
    L.mx_quantize_nvfp.argtypes = [_vp, _i32, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp]
    L.mx_dequantize_nvfp.restype = _i32
    L.mx_dequantize_nvfp.argtypes = [_vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _i32, _vp]
    L.mx_gemm_nvfp.restype = _i32
    L.mx_gemm_nvfp.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _i64, _i64, _i64, ctypes.c_float,
                               _vp, _i32, _i64, _vp]
    L.mx_norm_forward.restype = _i32
    L.mx_norm_forward.argtypes = [_vp, _i64, _vp, _i64, _i32, _i64, _i64, _i32, _vp, _vp, _i32, ctypes.c_float,
                                  _vp, _i64, _vp, _i64, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]
    L.mx_norm_backward.restype = _i32
    L.mx_norm_backward.argtypes = [_vp, _i64, _i32, _i64, _i64, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _i32, _vp,
                                   _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp]
    L.mx_norm_backward_workspace_bytes.restype = _i64
    L.mx_norm_backward_workspace_bytes.argtypes = [_i64, _i64]
    L.mx_glu_forward.restype = _i32
    L.mx_glu_forward.argtypes = [_vp, _i64, _vp, _i64, _i32, _i64, _i64, _i32, _vp, _i64, _i32, _i32, _vp, _vp,
                                 _i32, _vp, _vp, _vp, _vp, _vp]
    L.mx_glu_backward.restype = _i32
    L.mx_glu_backward.argtypes = [_vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _vp, _vp,
                                  _i32, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
    L.mx_glu_backward_dual_layout.restype = _i32
    L.mx_glu_backward_dual_layout.argtypes = [_vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp,
                                              _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp]
    L.mx_predict_workspace_bytes.restype = _i64
    L.mx_predict_workspace_bytes.argtypes = []
    L.mx_status_string.restype = ctypes.c_char_p
    L.mx_status_string.argtypes = [_i32]
    L.mx_last_error_message.restype = ctypes.c_char_p
    L.mx_last_error_message.argtypes = []
    _lib = L
    return L


def _status_name(s: int) -> str:
    try:
        return load().mx_status_string(s).decode()
    except Exception:
        return f"status {s}"


def _check(status: int):
    if status != MX_OK:
        raise MXError(status, load().mx_last_error_message().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# the handle of a device's current stream; torch.cuda.current_stream() builds
# an object around it (2.7 us against 0.1 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# torch.cuda.current_device() without its look at whether torch has started the GPU
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _other(stream) -> bool:
    """Whether a stream that a call was given is another than the current one."""
    if stream is None:
        return False
    at = _device()
    here = _raw_stream(at) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream != here or getattr(stream, "device_index", at) != at


def _run_on(stream, call, args):
    """call(**args) on the given stream, with what it allocates taken for that
    stream: torch hands memory out again in the order of the stream it was
    taken for, and a call's kernels are in the order of theirs.  New results
    are known to the caller's stream as well, where they may be dropped."""
    before = torch.cuda.current_stream()
    given = {id(a) for a in args.values()}
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        out = call(**{**args, "stream": None})
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and id(t) not in given:
            t.record_stream(before)
    return out


def _fmt(f) -> int:
    return FMTS[f] if isinstance(f, str) else int(f)


def elem_bits(fmt) -> int:
    return 4 if _fmt(fmt) == MX_E2M1 else 8


def qconfig(fmt, two_level=False, tscale_provided=False, sr=False, hadamard=False, seed=0,
            offset=0, block=32) -> mx_qconfig:
    return mx_qconfig(fmt=_fmt(fmt), block=block,
                      scale_fmt=MX_SCALE_E8M0_TENSOR_F32 if two_level else MX_SCALE_E8M0,
                      tscale=MX_TSCALE_PROVIDED if tscale_provided else MX_TSCALE_COMPUTE,
                      rounding=MX_SR if sr else MX_RNE, hadamard=int(bool(hadamard)),
                      seed=seed & 0xFFFFFFFFFFFFFFFF, offset=offset & 0xFFFFFFFF, reserved=0)


def _src(x: torch.Tensor):
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    if x.dtype == torch.float32:
        return MX_SRC_F32
    if x.dtype == torch.bfloat16:
        return MX_SRC_BF16
    raise TypeError("x must be float32 or bfloat16")


def copy_shapes(rows: int, cols: int, axis: int, fmt):
    """(codes shape, scales shape) of a stored copy."""
    bits = elem_bits(fmt)
    if axis == MX_AXIS_ROW:
        return (rows, cols * bits // 8), (rows, cols // 32)
    return (cols, rows * bits // 8), (cols, rows // 32)


def mx_quantize(x: torch.Tensor, axis: int, cfg: mx_qconfig, q: Optional[torch.Tensor] = None,
                scales: Optional[torch.Tensor] = None,
                tensor_scale: Optional[torch.Tensor] = None, stream=None
                ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    if (q is None or scales is None or tensor_scale is None) and _other(stream):
        return _run_on(stream, mx_quantize, locals())
    src = _src(x)
    rows, cols = x.shape
    qs, ss = copy_shapes(rows, cols, axis, cfg.fmt)
    if q is None:
        q = torch.empty(qs, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(ss, dtype=torch.uint8, device=x.device)
    if tensor_scale is None and cfg.scale_fmt == MX_SCALE_E8M0_TENSOR_F32:
        tensor_scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(load().mx_quantize(_ptr(x), src, rows, cols, x.stride(0), axis, ctypes.byref(cfg),
                              _ptr(q), _ptr(scales), _ptr(tensor_scale), _stream(stream)))
    return q, scales, tensor_scale


def mx_quantize_dual_layout(x: torch.Tensor, cfg: mx_qconfig, q_row=None, s_row=None,
                            q_col=None, s_col=None, tensor_scale=None, stream=None):
    if (q_row is None or s_row is None or q_col is None or s_col is None or tensor_scale is None) and _other(stream):
        return _run_on(stream, mx_quantize_dual_layout, locals())
    src = _src(x)
    rows, cols = x.shape
    qrs, srs = copy_shapes(rows, cols, MX_AXIS_ROW, cfg.fmt)
    qcs, scs = copy_shapes(rows, cols, MX_AXIS_COL, cfg.fmt)
    dev = x.device
    q_row = torch.empty(qrs, dtype=torch.uint8, device=dev) if q_row is None else q_row
    s_row = torch.empty(srs, dtype=torch.uint8, device=dev) if s_row is None else s_row
    q_col = torch.empty(qcs, dtype=torch.uint8, device=dev) if q_col is None else q_col
    s_col = torch.empty(scs, dtype=torch.uint8, device=dev) if s_col is None else s_col
    if tensor_scale is None and cfg.scale_fmt == MX_SCALE_E8M0_TENSOR_F32:
        tensor_scale = torch.empty(1, dtype=torch.float32, device=dev)
    _check(load().mx_quantize_dual_layout(_ptr(x), src, rows, cols, x.stride(0),
                                          ctypes.byref(cfg), _ptr(q_row), _ptr(s_row),
                                          _ptr(q_col), _ptr(s_col), _ptr(tensor_scale),
                                          _stream(stream)))
    return q_row, s_row, q_col, s_col, tensor_scale


def mx_gemm(qa, sa, ta, fa, qb, sb, tb, fb, M: int, N: int, K: int, alpha: float = 1.0,
            hadamard_k: bool = False, out_dtype: int = MX_OUT_BF16, c=None, ldc=None,
            stream=None) -> torch.Tensor:
    if c is None and _other(stream):
        return _run_on(stream, mx_gemm, locals())
    if c is None:
        c = torch.empty((M, N), dtype=torch.float32 if out_dtype == MX_OUT_F32 else torch.bfloat16,
                        device=qa.device)
    ldc = c.stride(0) if ldc is None else ldc
    _check(load().mx_gemm(_ptr(qa), _ptr(sa), _ptr(ta), _fmt(fa), _ptr(qb), _ptr(sb), _ptr(tb),
                          _fmt(fb), M, N, K, float(alpha), int(bool(hadamard_k)), _ptr(c),
                          out_dtype, ldc, _stream(stream)))
    return c


def mx_gemm_quantized(qa, sa, ta, fa, qb, sb, tb, fb, M: int, N: int, K: int, out_fmt="e4m3",
                      alpha: float = 1.0, hadamard_k: bool = False, qc=None, sc=None, stream=None):
    """GEMM with the output written as MX codes [M][N] and E8M0 scales [M][N/32]."""
    if (qc is None or sc is None) and _other(stream):
        return _run_on(stream, mx_gemm_quantized, locals())
    if qc is None:
        qc = torch.empty((M, N), dtype=torch.uint8, device=qa.device)
    if sc is None:
        sc = torch.empty((M, N // 32), dtype=torch.uint8, device=qa.device)
    _check(load().mx_gemm_quantized(_ptr(qa), _ptr(sa), _ptr(ta), _fmt(fa), _ptr(qb), _ptr(sb), _ptr(tb),
                                    _fmt(fb), M, N, K, float(alpha), int(bool(hadamard_k)), _fmt(out_fmt),
                                    _ptr(qc), _ptr(sc), _stream(stream)))
    return qc, sc


def mx_predict_tensor_scale(w: torch.Tensor, g: torch.Tensor, lr: float, fmt,
                            work: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """Predicted per-tensor scale of the next step's weights (weight auto-scaling)."""
    if _other(stream):
        return _run_on(stream, mx_predict_tensor_scale, locals())
    src = _src(w)
    if _src(g) != src or tuple(g.shape) != tuple(w.shape):
        raise ValueError("w and g must have the same dtype and shape")
    rows, cols = w.shape
    nbytes = int(load().mx_predict_workspace_bytes())
    if work is None:
        work = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    if scale_out is None:
        scale_out = torch.empty(1, dtype=torch.float32, device=w.device)
    _check(load().mx_predict_tensor_scale(_ptr(w), w.stride(0), _ptr(g), g.stride(0), src, rows, cols,
                                          float(lr), _fmt(fmt), _ptr(work), work.numel() * work.element_size(),
                                          _ptr(scale_out), _stream(stream)))
    return scale_out


def mx_predict_tensor_scale_noalloc(w: torch.Tensor, g: torch.Tensor, lr: float, fmt,
                                    scale_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """mx_predict_tensor_scale without a workspace: the library's per-GPU
    scratch holds the partial maxima (calls overlapping on one GPU race)."""
    if scale_out is None and _other(stream):
        return _run_on(stream, mx_predict_tensor_scale_noalloc, locals())
    src = _src(w)
    if _src(g) != src or tuple(g.shape) != tuple(w.shape):
        raise ValueError("w and g must have the same dtype and shape")
    rows, cols = w.shape
    if scale_out is None:
        scale_out = torch.empty(1, dtype=torch.float32, device=w.device)
    _check(load().mx_predict_tensor_scale_noalloc(_ptr(w), w.stride(0), _ptr(g), g.stride(0), src, rows, cols,
                                                  float(lr), _fmt(fmt), _ptr(scale_out), _stream(stream)))
    return scale_out


def mx_dequantize(q, scales, tensor_scale, fmt, rows: int, cols: int, axis: int,
                  hadamard: bool = False, out_dtype: int = MX_OUT_F32, out=None,
                  stream=None) -> torch.Tensor:
    if out is None and _other(stream):
        return _run_on(stream, mx_dequantize, locals())
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32 if out_dtype == MX_OUT_F32 else torch.bfloat16,
                          device=q.device)
    _check(load().mx_dequantize(_ptr(q), _ptr(scales), _ptr(tensor_scale), _fmt(fmt), rows, cols,
                                axis, int(bool(hadamard)), _ptr(out), out_dtype, _stream(stream)))
    return out


def mx_quantize_optstate(x: torch.Tensor, fmt="e4m3", group: int = 128, q=None, amax=None, kexp=None,
                         stream=None):
    """FP8 codes of an fp32 optimizer state after the per-group dynamic
    range expansion; returns (q uint8 [n], amax fp32 [n/group], k fp32 [n/group])."""
    if (q is None or amax is None or kexp is None) and _other(stream):
        return _run_on(stream, mx_quantize_optstate, locals())
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise TypeError("x must be a contiguous float32 tensor")
    n = x.numel()
    dev = x.device
    q = torch.empty(n, dtype=torch.uint8, device=dev) if q is None else q
    amax = torch.empty(n // group, dtype=torch.float32, device=dev) if amax is None else amax
    kexp = torch.empty(n // group, dtype=torch.float32, device=dev) if kexp is None else kexp
    _check(load().mx_quantize_optstate(_ptr(x), n, group, _fmt(fmt), _ptr(q), _ptr(amax), _ptr(kexp),
                                       _stream(stream)))
    return q, amax, kexp


def mx_dequantize_optstate(q, amax, kexp, fmt="e4m3", group: int = 128, out=None, stream=None) -> torch.Tensor:
    if out is None and _other(stream):
        return _run_on(stream, mx_dequantize_optstate, locals())
    n = q.numel()
    out = torch.empty(n, dtype=torch.float32, device=q.device) if out is None else out
    _check(load().mx_dequantize_optstate(_ptr(q), _ptr(amax), _ptr(kexp), n, group, _fmt(fmt), _ptr(out),
                                         _stream(stream)))
    return out


def nvfp_shapes(rows: int, cols: int, axis: int, local: bool):
    """(codes, block scales, second-level scales) shapes of an nvfp copy."""
    SR, L = (rows, cols) if axis == MX_AXIS_ROW else (cols, rows)
    return (SR, L // 2), (SR, L // 16), ((SR + NV_PANEL - 1) // NV_PANEL if local else 1,)


def mx_quantize_nvfp(x: torch.Tensor, axis: int = MX_AXIS_ROW, local: bool = False, q=None, scales=None,
                     tscale=None, stream=None):
    """NVFP4 copy of x with a global (local=False) or per-32-row-panel
    (local=True) second-level scale; returns (q, scales, tscale)."""
    if (q is None or scales is None or tscale is None) and _other(stream):
        return _run_on(stream, mx_quantize_nvfp, locals())
    src = _src(x)
    rows, cols = x.shape
    qs, ss, ts = nvfp_shapes(rows, cols, axis, local)
    dev = x.device
    q = torch.empty(qs, dtype=torch.uint8, device=dev) if q is None else q
    scales = torch.empty(ss, dtype=torch.uint8, device=dev) if scales is None else scales
    tscale = torch.empty(ts, dtype=torch.float32, device=dev) if tscale is None else tscale
    _check(load().mx_quantize_nvfp(_ptr(x), src, rows, cols, x.stride(0), axis, int(bool(local)), _ptr(q),
                                   _ptr(scales), _ptr(tscale), _stream(stream)))
    return q, scales, tscale


def mx_dequantize_nvfp(q, scales, tscale, rows: int, cols: int, axis: int = MX_AXIS_ROW, local: bool = False,
                       out_dtype: int = MX_OUT_F32, out=None, stream=None) -> torch.Tensor:
    if out is None and _other(stream):
        return _run_on(stream, mx_dequantize_nvfp, locals())
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32 if out_dtype == MX_OUT_F32 else torch.bfloat16,
                          device=q.device)
    _check(load().mx_dequantize_nvfp(_ptr(q), _ptr(scales), _ptr(tscale), rows, cols, axis, int(bool(local)),
                                     _ptr(out), out_dtype, _stream(stream)))
    return out


def mx_gemm_nvfp(qa, sa, ta, local_a: bool, qb, sb, tb, local_b: bool, M: int, N: int, K: int,
                 alpha: float = 1.0, out_dtype: int = MX_OUT_BF16, c=None, ldc=None, stream=None) -> torch.Tensor:
    if c is None and _other(stream):
        return _run_on(stream, mx_gemm_nvfp, locals())
    if c is None:
        c = torch.empty((M, N), dtype=torch.float32 if out_dtype == MX_OUT_F32 else torch.bfloat16,
                        device=qa.device)
    ldc = c.stride(0) if ldc is None else ldc
    _check(load().mx_gemm_nvfp(_ptr(qa), _ptr(sa), _ptr(ta), int(bool(local_a)), _ptr(qb), _ptr(sb), _ptr(tb),
                               int(bool(local_b)), M, N, K, float(alpha), _ptr(c), out_dtype, ldc, _stream(stream)))
    return c


# ---------------------------------------------------------------------------
# activation operators (norm, gated activation) with 8-bit checkpoints
# ---------------------------------------------------------------------------
class Checkpoint(NamedTuple):
    """An MX row copy kept for the backward pass: element format, codes
    [rows][cols] and scale bytes [rows][cols / 32] (uint8, dense)."""
    fmt: int
    q: torch.Tensor
    s: torch.Tensor


class NormForward(NamedTuple):
    y: Optional[torch.Tensor]
    sum: Optional[torch.Tensor]
    qy: Optional[torch.Tensor]
    sy: Optional[torch.Tensor]
    qx: Optional[torch.Tensor]
    sx: Optional[torch.Tensor]
    mean: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


class NormBackward(NamedTuple):
    dx: torch.Tensor
    dweight: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


class GluForward(NamedTuple):
    h: Optional[torch.Tensor]
    qh: Optional[torch.Tensor]
    sh: Optional[torch.Tensor]
    qg: Optional[torch.Tensor]
    sg: Optional[torch.Tensor]
    qu: Optional[torch.Tensor]
    su: Optional[torch.Tensor]


class GluBackward(NamedTuple):
    dgate: torch.Tensor
    dup: torch.Tensor
    h: Optional[torch.Tensor]


class GluBackwardDual(NamedTuple):
    q_row: torch.Tensor
    s_row: torch.Tensor
    q_col: torch.Tensor
    s_col: torch.Tensor
    qh_col: Optional[torch.Tensor]
    sh_col: Optional[torch.Tensor]


def checkpoint(fmt, q: torch.Tensor, s: torch.Tensor) -> Checkpoint:
    """Codes and scales as mx_quantize (MX_AXIS_ROW) or a forward call wrote them."""
    return Checkpoint(_fmt(fmt), q, s)


def _misfit(t: torch.Tensor, shape, dtype, at: int, name: str, layout: str):
    """Why t is not what a call needs."""
    if t.get_device() != at:
        return ValueError(f"{name} must be on the device of the call's first tensor")
    if t.dtype is not dtype:
        return TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        return ValueError(f"{name} must have shape {tuple(shape)}")
    return ValueError(f"{name} must {layout}")


# The checks below run on every call, so each looks at a tensor once and
# returns what the call passes on.

def _matrix(t: torch.Tensor, shape, dtype, at: int, name: str):
    """(address, row stride in elements) of a matrix of this shape, type and device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == at:
        ld, unit = t.stride()
        rows, cols = shape
        if unit == 1 or cols <= 1:
            return t.data_ptr(), ld if rows > 1 or ld > cols else cols    # one row: any stride will do
    raise _misfit(t, shape, dtype, at, name, "have unit column stride")


def _maybe_matrix(t: Optional[torch.Tensor], shape, dtype, at: int, name: str):
    return (None, 0) if t is None else _matrix(t, shape, dtype, at, name)


def _dense(t: torch.Tensor, shape, dtype, at: int, name: str) -> int:
    """Address of a contiguous tensor of this shape, type and device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == at and t.is_contiguous():
        return t.data_ptr()
    raise _misfit(t, shape, dtype, at, name, "be contiguous")


def _first(x: torch.Tensor, name: str):
    """(source code, shape, type, device, address, row stride) of a call's first operand."""
    shape, dtype, at = x.shape, x.dtype, x.get_device()
    if len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    if dtype is torch.bfloat16:
        src = MX_SRC_BF16
    elif dtype is torch.float32:
        src = MX_SRC_F32
    else:
        raise TypeError(f"{name} must be float32 or bfloat16")
    return (src, shape, dtype, at, *_matrix(x, shape, dtype, at, name))


# What a call writes: the caller's tensor, looked at as above, or a new one,
# which needs no looking at.  (A new one costs 1.2 us by empty_like and 1.4 by
# new_empty_strided; new_empty, which first works out the strides, 1.6-1.8.)

def _out_matrix(t: Optional[torch.Tensor], first: torch.Tensor, shape, dtype, at: int, name: str):
    """(tensor, address, row stride) of a matrix output of the first operand's shape."""
    if t is None:
        t = torch.empty_like(first, dtype=dtype)
        return t, t.data_ptr(), shape[1]
    return (t, *_matrix(t, shape, dtype, at, name))


def _out_vector(t: Optional[torch.Tensor], first: torch.Tensor, n: int, at: int, name: str):
    """(tensor, address) of a float32 vector output."""
    if t is None:
        t = first.new_empty_strided((n,), (1,), dtype=torch.float32)
        return t, t.data_ptr()
    return t, _dense(t, (n,), torch.float32, at, name)


def _out_bytes(t: Optional[torch.Tensor], first: torch.Tensor, shape, at: int, name: str):
    """(tensor, address) of codes or scales."""
    if t is None:
        t = first.new_empty_strided(shape, (shape[1], 1), dtype=torch.uint8)
        return t, t.data_ptr()
    return t, _dense(t, shape, torch.uint8, at, name)


def _out_dtype(dtype, default):
    """(torch dtype, MX_OUT_* code) of a matrix output."""
    dtype = default if dtype is None else dtype
    if dtype is torch.bfloat16:
        return dtype, MX_OUT_BF16
    if dtype is torch.float32:
        return dtype, MX_OUT_F32
    raise TypeError("out_dtype must be float32 or bfloat16")


def _copy_out(fmt, q, s, shape, first, at, names):
    """(format code, codes, scales, their addresses) of a row copy to be
    written, new where the caller gave none; nothing without a format.
    first: the call's first tensor."""
    if fmt is None:
        if q is not None or s is not None:
            raise ValueError(f"{names[0]} need a format")
        return 0, None, None, None, None
    q, pq = _out_bytes(q, first, shape, at, names[0])
    s, ps = _out_bytes(s, first, (shape[0], shape[1] // 32), at, names[1])
    return _fmt(fmt), q, s, pq, ps


def _copy_in(c: Optional[Checkpoint], shape, at: int, names):
    """(format code, addresses of codes and scales) of a checkpoint that is read."""
    if c is None:
        return 0, None, None
    rows, cols = shape
    return (c.fmt, _dense(c.q, shape, torch.uint8, at, names[0]),
            _dense(c.s, (rows, cols // 32), torch.uint8, at, names[1]))


_Y, _X = ("the codes of y", "the scales of y"), ("the checkpoint's codes", "the checkpoint's scales")
_H = ("the codes of h", "the scales of h")
_GATE = ("the codes of gate's checkpoint", "the scales of gate's checkpoint")
_UP = ("the codes of up's checkpoint", "the scales of up's checkpoint")
_ROW = ("the codes of the row copy", "the scales of the row copy")
_COL = ("the codes of the column copy", "the scales of the column copy")


def _params(weight, bias, cols: int, at: int):
    """(addresses, common dtype code) of the parameters."""
    given = weight if weight is not None else bias
    if given is None:
        return None, None, 0
    dtype = given.dtype
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise TypeError("weight and bias must be float32 or bfloat16")
    return (None if weight is None else _dense(weight, (cols,), dtype, at, "weight"),
            None if bias is None else _dense(bias, (cols,), dtype, at, "bias"),
            MX_SRC_F32 if dtype is torch.float32 else MX_SRC_BF16)


def _stream_on(stream, at: int) -> int:
    """The given stream, or the current one."""
    if at < 0 or at != _device():
        raise ValueError("the tensors must be on the current GPU")
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(at) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def mx_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                    eps: float = 1e-5, kind: str = "rms", residual: Optional[torch.Tensor] = None,
                    write_y: bool = True, out_dtype: Optional[torch.dtype] = None, y_fmt=None, ckpt_fmt=None,
                    stats: bool = True, sum_out=None, y=None, qy=None, sy=None, qx=None, sx=None, mean=None,
                    rstd=None, stream=None) -> NormForward:
    """RMS norm or layer norm of x (+ residual), with y as a tensor, as an MX
    row copy (y_fmt) or both, and the 8-bit checkpoint (ckpt_fmt) of what was
    normalised.  stats: also mean (layer norm) and rstd for the backward."""
    if _other(stream):
        return _run_on(stream, mx_norm_forward, locals())
    src, shape, dtype, at, px, ld_x = _first(x, "x")
    rows, cols = shape
    k = NORMS[kind]
    pres = psum = py = None
    ld_res = ld_sum = ld_y = 0
    if residual is not None:
        pres, ld_res = _matrix(residual, shape, dtype, at, "residual")
        sum_out, psum, ld_sum = _out_matrix(sum_out, x, shape, dtype, at, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    out_dtype, out = _out_dtype(out_dtype, dtype)
    if write_y:
        y, py, ld_y = _out_matrix(y, x, shape, out_dtype, at, "y")
    else:
        y = None
    yf, qy, sy, pqy, psy = _copy_out(y_fmt, qy, sy, shape, x, at, _Y)
    cf, qx, sx, pqx, psx = _copy_out(ckpt_fmt, qx, sx, shape, x, at, _X)
    pw, pb, pd = _params(weight, bias, cols, at)
    pmean = prstd = None
    if stats:
        rstd, prstd = _out_vector(rstd, x, rows, at, "rstd")
    else:
        rstd = None
    if stats and k == MX_NORM_LAYER:
        mean, pmean = _out_vector(mean, x, rows, at, "mean")
    else:
        mean = None
    _check(load().mx_norm_forward(px, ld_x, pres, ld_res, src, rows, cols, k, pw, pb, pd, eps, psum, ld_sum, py,
                                  ld_y, out, yf, pqy, psy, cf, pqx, psx, pmean, prstd, _stream_on(stream, at)))
    return NormForward(y, sum_out, qy, sy, qx, sx, mean, rstd)


def mx_norm_backward(dy: torch.Tensor, rstd: torch.Tensor, x: Optional[torch.Tensor] = None,
                     ckpt: Optional[Checkpoint] = None, mean: Optional[torch.Tensor] = None,
                     weight: Optional[torch.Tensor] = None, kind: str = "rms",
                     dsum: Optional[torch.Tensor] = None, want_dweight: bool = True, want_dbias: bool = False,
                     dx=None, dweight=None, dbias=None, work=None, stream=None) -> NormBackward:
    """Gradients of mx_norm_forward from what it normalised (x) or from its
    checkpoint; dsum is a gradient of the same tensor from elsewhere, added
    to dx.  dweight and dbias are float32."""
    if _other(stream):
        return _run_on(stream, mx_norm_backward, locals())
    src, shape, dtype, at, pdy, ld_dy = _first(dy, "dy")
    rows, cols = shape
    k = NORMS[kind]
    px, ld_x = _maybe_matrix(x, shape, dtype, at, "x")
    cf, pqx, psx = _copy_in(ckpt, shape, at, _X)
    prstd = _dense(rstd, (rows,), torch.float32, at, "rstd")
    pmean = _dense(mean, (rows,), torch.float32, at, "mean") if k == MX_NORM_LAYER and mean is not None else None
    pds, ld_ds = _maybe_matrix(dsum, shape, dtype, at, "dsum")
    dx, pdx, ld_dx = _out_matrix(dx, dy, shape, dtype, at, "dx")
    pw, _, pd = _params(weight, None, cols, at)
    pdw = pdb = pwork = None
    nbytes = 0
    L = load()
    if want_dweight:
        dweight, pdw = _out_vector(dweight, dy, cols, at, "dweight")
    else:
        dweight = None
    if want_dbias:
        dbias, pdb = _out_vector(dbias, dy, cols, at, "dbias")
    else:
        dbias = None
    if want_dweight or want_dbias:
        if work is None:
            nbytes = L.mx_norm_backward_workspace_bytes(rows, cols)
            work = dy.new_empty_strided((nbytes,), (1,), dtype=torch.uint8)
        elif work.get_device() != at or not work.is_contiguous():
            raise ValueError("work must be contiguous and on the device of dy")
        else:
            nbytes = work.numel() * work.element_size()
        pwork = work.data_ptr()
    _check(L.mx_norm_backward(pdy, ld_dy, src, rows, cols, px, ld_x, cf, pqx, psx, pmean, prstd, k, pw, pd, pds,
                              ld_ds, pdx, ld_dx, pdw, pdb, pwork, nbytes, _stream_on(stream, at)))
    return NormBackward(dx, dweight, dbias)


def mx_glu_forward(gate: torch.Tensor, up: torch.Tensor, act: str = "silu", write_h: bool = True,
                   out_dtype: Optional[torch.dtype] = None, h_fmt=None, ckpt_fmt=None, h=None, qh=None, sh=None,
                   qg=None, sg=None, qu=None, su=None, stream=None) -> GluForward:
    """h = act(gate) * up as a tensor, as an MX row copy (h_fmt) or both, and
    the 8-bit checkpoints (ckpt_fmt) of gate and up."""
    if _other(stream):
        return _run_on(stream, mx_glu_forward, locals())
    src, shape, dtype, at, pg, ld_g = _first(gate, "gate")
    rows, cols = shape
    pu, ld_u = _matrix(up, shape, dtype, at, "up")
    out_dtype, out = _out_dtype(out_dtype, dtype)
    if write_h:
        h, ph, ld_h = _out_matrix(h, gate, shape, out_dtype, at, "h")
    else:
        h, ph, ld_h = None, None, 0
    hf, qh, sh, pqh, psh = _copy_out(h_fmt, qh, sh, shape, gate, at, _H)
    cf, qg, sg, pqg, psg = _copy_out(ckpt_fmt, qg, sg, shape, gate, at, _GATE)
    _, qu, su, pqu, psu = _copy_out(ckpt_fmt, qu, su, shape, gate, at, _UP)
    _check(load().mx_glu_forward(pg, ld_g, pu, ld_u, src, rows, cols, ACTS[act], ph, ld_h, out, hf, pqh, psh, cf,
                                 pqg, psg, pqu, psu, _stream_on(stream, at)))
    return GluForward(h, qh, sh, qg, sg, qu, su)


def _glu_inputs(dh, gate, up, gate_ckpt, up_ckpt, act):
    """Shape, type and device of the backward calls' operands, and their shared leading arguments."""
    src, shape, dtype, at, pd, ld_d = _first(dh, "dh")
    gf, pqg, psg = _copy_in(gate_ckpt, shape, at, _GATE)
    uf, pqu, psu = _copy_in(up_ckpt, shape, at, _UP)
    if gate_ckpt is not None and up_ckpt is not None and gf != uf:
        raise ValueError("the checkpoints of gate and up must have one format")
    return shape, dtype, at, (pd, ld_d, src, *shape, *_maybe_matrix(gate, shape, dtype, at, "gate"),
                              *_maybe_matrix(up, shape, dtype, at, "up"), gf, pqg, psg, pqu, psu, ACTS[act])


def mx_glu_backward(dh: torch.Tensor, gate: Optional[torch.Tensor] = None, up: Optional[torch.Tensor] = None,
                    act: str = "silu", gate_ckpt: Optional[Checkpoint] = None,
                    up_ckpt: Optional[Checkpoint] = None, recompute_h: bool = False, dgate=None, dup=None, h=None,
                    stream=None) -> GluBackward:
    """Gradients of mx_glu_forward from gate and up, or from their
    checkpoints; recompute_h: also h = act(gate) * up."""
    if _other(stream):
        return _run_on(stream, mx_glu_backward, locals())
    shape, dtype, at, head = _glu_inputs(dh, gate, up, gate_ckpt, up_ckpt, act)
    dgate, pdg, ld_dg = _out_matrix(dgate, dh, shape, dtype, at, "dgate")
    dup, pdu, ld_du = _out_matrix(dup, dh, shape, dtype, at, "dup")
    if recompute_h:
        h, ph, ld_h = _out_matrix(h, dh, shape, dtype, at, "h")
    else:
        h, ph, ld_h = None, None, 0
    _check(load().mx_glu_backward(*head, pdg, ld_dg, pdu, ld_du, ph, ld_h, _stream_on(stream, at)))
    return GluBackward(dgate, dup, h)


def mx_glu_backward_dual_layout(dh: torch.Tensor, gate: Optional[torch.Tensor] = None,
                                up: Optional[torch.Tensor] = None, act: str = "silu",
                                gate_ckpt: Optional[Checkpoint] = None, up_ckpt: Optional[Checkpoint] = None,
                                fmt="e5m2", h_fmt=None, q_row=None, s_row=None, q_col=None, s_col=None,
                                qh_col=None, sh_col=None, stream=None) -> GluBackwardDual:
    """mx_glu_backward straight into the backward GEMMs' operands: the row and
    column copies of [dgate | dup] and (h_fmt) the column copy of h."""
    if _other(stream):
        return _run_on(stream, mx_glu_backward_dual_layout, locals())
    shape, _, at, head = _glu_inputs(dh, gate, up, gate_ckpt, up_ckpt, act)
    rows, cols = shape
    f, q_row, s_row, pqr, psr = _copy_out(fmt, q_row, s_row, (rows, 2 * cols), dh, at, _ROW)
    _, q_col, s_col, pqc, psc = _copy_out(fmt, q_col, s_col, (2 * cols, rows), dh, at, _COL)
    hf, qh_col, sh_col, pqh, psh = _copy_out(h_fmt, qh_col, sh_col, (cols, rows), dh, at, _H)
    _check(load().mx_glu_backward_dual_layout(*head, f, pqr, psr, pqc, psc, hf, pqh, psh, _stream_on(stream, at)))
    return GluBackwardDual(q_row, s_row, q_col, s_col, qh_col, sh_col)
