"""Python binding of libhqq (include/hqq.h): HQQ group-wise weight-only
quantization of fp16 weight matrices on NVIDIA B200 (sm_100a).

Argument marshalling only: every step of the quantization and dequantization
runs in libhqq's CUDA kernels.  torch supplies device memory and the current
stream.  There is no fallback: importing fails loudly when libhqq.so is absent,
and every call raises ``HQQError`` on a non-zero status.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

__all__ = ["HQQError", "hqq_quantize", "hqq_quantize_ex", "hqq_quantize_half", "hqq_dequantize",
           "hqq_packed_bytes", "hqq_status_string", "QuantizedMatrix", "LIB_PATH",
           "Meta8", "hqq_meta_groups", "hqq_meta_quantize", "hqq_meta_quantize_batch",
           "hqq_meta_dequantize",
           "hqq_dequantize_meta", "hqq_linear", "hqq_linear_meta", "hqq_lowrank", "hqq_distill",
           "Adapters", "hqq_linear_adapters", "hqq_linear_adapters_backward",
           "DEFAULT_P", "DEFAULT_BETA", "DEFAULT_KAPPA", "DEFAULT_ITERS"]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhqq.so")

DEFAULT_P, DEFAULT_BETA, DEFAULT_KAPPA, DEFAULT_ITERS = 0.7, 1.0, 1.01, 20

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python weight_only_quantization_b200/build.py`")

_lib = ctypes.CDLL(LIB_PATH)
_P, _I64, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_lib.hqq_packed_bytes.argtypes = [_I64, _I64, _I]
_lib.hqq_packed_bytes.restype = _I64
_lib.hqq_status_string.argtypes = [_I]
_lib.hqq_status_string.restype = ctypes.c_char_p
_lib.hqq_quantize.argtypes = [_P, _I64, _I64, _I, _I, _F, _F, _F, _I, _P, _P, _P, _P]
_lib.hqq_quantize.restype = _I
_lib.hqq_quantize_ex.argtypes = [_P, _I64, _I64, _I, _I, _F, _F, _F, _I, _P, _P, _P, _P, _P, _P,
                                 _P]
_lib.hqq_quantize_ex.restype = _I
_lib.hqq_quantize_half.argtypes = [_P, _I64, _I64, _I, _I, _F, _F, _F, _I, _P, _P, _P, _P, _P, _P,
                                   _P, _P]
_lib.hqq_quantize_half.restype = _I
_lib.hqq_dequantize.argtypes = [_P, _P, _P, _I64, _I64, _I, _I, _P, _P]
_lib.hqq_dequantize.restype = _I
_lib.hqq_meta_groups.argtypes = [_I64, _I64]
_lib.hqq_meta_groups.restype = _I64
_lib.hqq_meta_quantize.argtypes = [_P, _I64, _I64, _P, _P, _P, _P]
_lib.hqq_meta_quantize.restype = _I
_lib.hqq_meta_dequantize.argtypes = [_P, _P, _P, _I64, _I64, _P, _P]
_lib.hqq_meta_dequantize.restype = _I


class _CMeta8(ctypes.Structure):
    """struct hqq_meta8 of include/hqq.h."""
    _fields_ = [("codes", _P), ("scale", _P), ("zero", _P), ("group", _I64)]


class _CMetaJob(ctypes.Structure):
    """struct hqq_meta_job of include/hqq.h."""
    _fields_ = [("x", _P), ("n", _I64), ("mgroup", _I64), ("codes", _P), ("scale", _P),
                ("zero", _P)]


_lib.hqq_meta_quantize_batch.argtypes = [ctypes.POINTER(_CMetaJob), _I64, _P]
_lib.hqq_meta_quantize_batch.restype = _I
_lib.hqq_dequantize_meta.argtypes = [_P, ctypes.POINTER(_CMeta8), _P, ctypes.POINTER(_CMeta8),
                                     _I64, _I64, _I, _I, _P, _P]
_lib.hqq_dequantize_meta.restype = _I
_lib.hqq_linear.argtypes = [_P, _I64, _P, _P, _P, _I64, _I64, _I, _I, _P, _P, _P]
_lib.hqq_linear.restype = _I
_lib.hqq_linear_meta.argtypes = [_P, _I64, _P, ctypes.POINTER(_CMeta8), _P,
                                 ctypes.POINTER(_CMeta8), _I64, _I64, _I, _I, _P, _P, _P]
_lib.hqq_linear_meta.restype = _I
_lib.hqq_lowrank_workspace_bytes.argtypes = [_I64, _I64, _I]
_lib.hqq_lowrank_workspace_bytes.restype = _I64
_lib.hqq_lowrank.argtypes = [_P, _P, _P, _P, _I64, _I64, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P,
                             _I64, _P]
_lib.hqq_lowrank.restype = _I


class _CAdapters(ctypes.Structure):
    """struct hqq_adapters of include/hqq.h."""
    _fields_ = [("A", _P), ("B", _P), ("scaling", _P), ("A_stride", _I64), ("B_stride", _I64),
                ("count", _I), ("rank", _I), ("dtype", _I)]


_lib.hqq_linear_adapters_workspace_bytes.argtypes = [_I64, _I64, _I64, _I, _I, _I]
_lib.hqq_linear_adapters_workspace_bytes.restype = _I64
_lib.hqq_linear_adapters.argtypes = [_P, _I64, _P, _P, _P, ctypes.POINTER(_CMeta8),
                                     ctypes.POINTER(_CMeta8), _I64, _I64, _I, _I,
                                     ctypes.POINTER(_CAdapters), _P, _P, _P, _P, _I64, _P]
_lib.hqq_linear_adapters.restype = _I
_lib.hqq_linear_adapters_backward.argtypes = [_P, _P, _I64, _P, _P, _P, ctypes.POINTER(_CMeta8),
                                              ctypes.POINTER(_CMeta8), _I64, _I64, _I, _I,
                                              ctypes.POINTER(_CAdapters), _P, _P, _P, _P, _P, _P,
                                              _I64, _P]
_lib.hqq_linear_adapters_backward.restype = _I
_lib.hqq_distill.argtypes = [_P, _I64, _I, _I64, _I64, _P, _I, _P, _I, _I64, _F, _P, _P, _P, _P,
                             _P, _I64, _P]
_lib.hqq_distill.restype = _I


class HQQError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(hqq_status_string(status))


def hqq_status_string(status: int) -> str:
    return _lib.hqq_status_string(status).decode()


def hqq_packed_bytes(rows: int, cols: int, nbits: int) -> int:
    n = _lib.hqq_packed_bytes(rows, cols, nbits)
    if n < 0:
        raise HQQError(2 if nbits in (1, 2, 3, 4, 8) else 3)
    return int(n)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(st: int):
    if st != 0:
        raise HQQError(st)


@dataclass
class QuantizedMatrix:
    """Packed codes + fp16 scale/zero of one [rows, cols] matrix."""
    packed: "torch.Tensor"     # uint8 [hqq_packed_bytes]
    scale: "torch.Tensor"      # fp16 [rows, cols/group]
    zero: "torch.Tensor"       # fp16 [rows, cols/group]
    rows: int
    cols: int
    nbits: int
    group: int
    zero_f32: "torch.Tensor | None" = None
    iters: "torch.Tensor | None" = None
    err: "torch.Tensor | None" = None
    half: "torch.Tensor | None" = None      # uint8: group solved in half precision


def _tensors(result):
    """The tensors of what a call returns."""
    if isinstance(result, (tuple, list)):
        for r in result:
            yield from _tensors(r)
    elif isinstance(result, (QuantizedMatrix, Meta8)):
        yield from _tensors(list(vars(result).values()))
    elif hasattr(result, "record_stream"):
        yield result


def _on(stream, on, call, *args):
    """call(*args) with ``stream`` as the current one (``on``: a tensor of the call).  The
    allocator hands out and takes back memory in the order of one stream's work, so what
    the call allocates has to be taken in that of its launches; results made there are,
    once freed, not handed out before the work of that time on the stream that the caller
    is on has ended."""
    import torch
    if on.is_cuda and not hasattr(stream, "device"):     # (any object that has a handle)
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=on.device)
    if not on.is_cuda or on.get_device() != stream.device.index:
        raise ValueError("stream must be on the tensors' device")
    current = torch.cuda.current_stream(stream.device)
    if stream == current:
        return call(*args)
    with torch.cuda.stream(stream):
        out = call(*args)
    for t in _tensors(out):
        if not any(t is a for a in args):
            t.record_stream(current)
    return out


def _outputs(W, nbits, group, packed, scale, zero):
    import torch
    rows, cols = W.shape
    if packed is None:
        packed = torch.empty(hqq_packed_bytes(rows, cols, nbits), dtype=torch.uint8,
                             device=W.device)
    meta = (rows, cols // group if group > 0 else 0)
    if scale is None:
        scale = torch.empty(meta, dtype=torch.float16, device=W.device)
    if zero is None:
        zero = torch.empty(meta, dtype=torch.float16, device=W.device)
    return packed, scale, zero


def _check_tensor(t, name):
    if t is not None and not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def _precision(precision: str) -> bool:
    if precision not in ("fp32", "fp16"):
        raise ValueError("precision must be 'fp32' (single-precision solver) or 'fp16' "
                         "(the half-precision solver)")
    return precision == "fp16"


def hqq_quantize(W, nbits: int = 4, group: int = 64, p: float = DEFAULT_P,
                 beta: float = DEFAULT_BETA, kappa: float = DEFAULT_KAPPA,
                 iters: int = DEFAULT_ITERS, packed=None, scale=None, zero=None,
                 stream=None, precision: str = "fp32") -> QuantizedMatrix:
    """Quantize a contiguous fp16 CUDA matrix [rows, cols] (see include/hqq.h);
    ``precision="fp16"`` runs the half-precision solver (hqq_quantize_half)."""
    if stream is not None:
        return _on(stream, W, hqq_quantize, W, nbits, group, p, beta, kappa, iters, packed, scale,
                   zero, None, precision)
    import torch
    if W.dtype != torch.float16 or W.dim() != 2:
        raise ValueError("W must be a 2-D float16 tensor")
    half = _precision(precision)
    for t, n in ((W, "W"), (packed, "packed"), (scale, "scale"), (zero, "zero")):
        _check_tensor(t, n)
    packed, scale, zero = _outputs(W, nbits, group, packed, scale, zero)
    rows, cols = W.shape
    if half:
        _check(_lib.hqq_quantize_half(_ptr(W), rows, cols, nbits, group, p, beta, kappa, iters,
                                      _ptr(packed), _ptr(scale), _ptr(zero), None, None, None,
                                      None, _stream()))
    else:
        _check(_lib.hqq_quantize(_ptr(W), rows, cols, nbits, group, p, beta, kappa, iters,
                                 _ptr(packed), _ptr(scale), _ptr(zero), _stream()))
    return QuantizedMatrix(packed, scale, zero, rows, cols, nbits, group)


def hqq_quantize_ex(W, nbits: int = 4, group: int = 64, p: float = DEFAULT_P,
                    beta: float = DEFAULT_BETA, kappa: float = DEFAULT_KAPPA,
                    iters: int = DEFAULT_ITERS, packed=None, scale=None, zero=None,
                    zero_f32=None, iters_out=None, err_out=None, stream=None,
                    precision: str = "fp32", half_out=None) -> QuantizedMatrix:
    """hqq_quantize plus the fp32 zero, the solver's l_p error and the
    accepted-iteration count of every group (and, with ``precision="fp16"``,
    which groups were solved in half precision)."""
    if stream is not None:
        return _on(stream, W, hqq_quantize_ex, W, nbits, group, p, beta, kappa, iters, packed,
                   scale, zero, zero_f32, iters_out, err_out, None, precision, half_out)
    import torch
    if W.dtype != torch.float16 or W.dim() != 2:
        raise ValueError("W must be a 2-D float16 tensor")
    half = _precision(precision)
    for t, n in ((W, "W"), (packed, "packed"), (scale, "scale"), (zero, "zero"),
                 (zero_f32, "zero_f32"), (iters_out, "iters_out"), (err_out, "err_out")):
        _check_tensor(t, n)
    packed, scale, zero = _outputs(W, nbits, group, packed, scale, zero)
    rows, cols = W.shape
    meta = (rows, cols // group if group > 0 else 0)
    if zero_f32 is None:
        zero_f32 = torch.empty(meta, dtype=torch.float32, device=W.device)
    if iters_out is None:
        iters_out = torch.empty(meta, dtype=torch.uint8, device=W.device)
    if err_out is None:
        err_out = torch.empty(meta, dtype=torch.float32, device=W.device)
    if half:
        _check_tensor(half_out, "half_out")
        if half_out is None:
            half_out = torch.empty(meta, dtype=torch.uint8, device=W.device)
        _check(_lib.hqq_quantize_half(_ptr(W), rows, cols, nbits, group, p, beta, kappa, iters,
                                      _ptr(packed), _ptr(scale), _ptr(zero), _ptr(zero_f32),
                                      _ptr(err_out), _ptr(iters_out), _ptr(half_out),
                                      _stream()))
    else:
        half_out = None
        _check(_lib.hqq_quantize_ex(_ptr(W), rows, cols, nbits, group, p, beta, kappa, iters,
                                    _ptr(packed), _ptr(scale), _ptr(zero), _ptr(zero_f32),
                                    _ptr(err_out), _ptr(iters_out), _stream()))
    return QuantizedMatrix(packed, scale, zero, rows, cols, nbits, group, zero_f32, iters_out,
                           err_out, half_out)


def hqq_dequantize(q: QuantizedMatrix, out=None, stream=None):
    """fp16 [rows, cols] = (code - zero) * scale  (see include/hqq.h)."""
    if stream is not None:
        return _on(stream, q.packed, hqq_dequantize, q, out)
    import torch
    for t, n in ((q.packed, "packed"), (q.scale, "scale"), (q.zero, "zero"), (out, "out")):
        _check_tensor(t, n)
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=torch.float16, device=q.packed.device)
    _check(_lib.hqq_dequantize(_ptr(q.packed), _ptr(q.scale), _ptr(q.zero), q.rows, q.cols,
                               q.nbits, q.group, _ptr(out), _stream()))
    return out


@dataclass
class Meta8:
    """8-bit form of a meta tensor (a matrix's zero points or scales)."""
    codes: "torch.Tensor"      # uint8 [n]
    scale: "torch.Tensor"      # fp16 [hqq_meta_groups(n, group)]
    zero: "torch.Tensor"       # fp16 [hqq_meta_groups(n, group)]
    group: int                 # 0 (one group) or a power of two

    def _c(self):
        return _CMeta8(self.codes.data_ptr(), self.scale.data_ptr(), self.zero.data_ptr(),
                       self.group)


def hqq_meta_groups(n: int, mgroup: int) -> int:
    g = _lib.hqq_meta_groups(n, mgroup)
    if g < 0:
        raise HQQError(2)
    return int(g)


def hqq_meta_quantize(x, mgroup: int = 0, codes=None, scale=None, zero=None,
                      stream=None) -> Meta8:
    """8-bit min-max round-to-nearest of an fp16 meta tensor (flat order;
    ``mgroup`` consecutive values per group, 0 = one group); see include/hqq.h."""
    if stream is not None:
        return _on(stream, x, hqq_meta_quantize, x, mgroup, codes, scale, zero)
    import torch
    if x.dtype != torch.float16:
        raise ValueError("x must be float16")
    _check_tensor(x, "x")
    n = x.numel()
    ng = hqq_meta_groups(n, mgroup)
    if codes is None:
        codes = torch.empty(n, dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(ng, dtype=torch.float16, device=x.device)
    if zero is None:
        zero = torch.empty(ng, dtype=torch.float16, device=x.device)
    for t, nm in ((codes, "codes"), (scale, "scale"), (zero, "zero")):
        _check_tensor(t, nm)
    _check(_lib.hqq_meta_quantize(_ptr(x), n, mgroup, _ptr(codes), _ptr(scale), _ptr(zero),
                                  _stream()))
    return Meta8(codes, scale, zero, mgroup)


def hqq_meta_quantize_batch(tensors, stream=None, outputs=None) -> list:
    """hqq_meta_quantize of many fp16 meta tensors in shared launches.
    ``tensors`` is a list of (x, mgroup); ``outputs`` optionally a list of
    Meta8 to write into (same order).  Returns the list of Meta8."""
    if stream is not None and tensors:
        return _on(stream, tensors[0][0], hqq_meta_quantize_batch, tensors, None, outputs)
    import torch
    out = []
    jobs = (_CMetaJob * max(len(tensors), 1))()
    for i, (x, mgroup) in enumerate(tensors):
        if x.dtype != torch.float16:
            raise ValueError("x must be float16")
        _check_tensor(x, "x")
        n = x.numel()
        if outputs is not None:
            m = outputs[i]
        else:
            ng = hqq_meta_groups(n, mgroup)
            m = Meta8(torch.empty(n, dtype=torch.uint8, device=x.device),
                      torch.empty(ng, dtype=torch.float16, device=x.device),
                      torch.empty(ng, dtype=torch.float16, device=x.device), mgroup)
        for t, nm in ((m.codes, "codes"), (m.scale, "scale"), (m.zero, "zero")):
            _check_tensor(t, nm)
        jobs[i] = _CMetaJob(x.data_ptr(), n, mgroup, m.codes.data_ptr(), m.scale.data_ptr(),
                            m.zero.data_ptr())
        out.append(m)
    _check(_lib.hqq_meta_quantize_batch(jobs, len(tensors), _stream()))
    return out


def hqq_meta_dequantize(m: Meta8, out=None, stream=None):
    """fp16 [n] = (code - zero) * scale per value of an 8-bit meta tensor."""
    if stream is not None:
        return _on(stream, m.codes, hqq_meta_dequantize, m, out)
    import torch
    for t, nm in ((m.codes, "codes"), (m.scale, "scale"), (m.zero, "zero"), (out, "out")):
        _check_tensor(t, nm)
    n = m.codes.numel()
    if out is None:
        out = torch.empty(n, dtype=torch.float16, device=m.codes.device)
    _check(_lib.hqq_meta_dequantize(_ptr(m.codes), _ptr(m.scale), _ptr(m.zero), n, m.group,
                                    _ptr(out), _stream()))
    return out


def hqq_dequantize_meta(packed, zero_q: Meta8, rows: int, cols: int, nbits: int, group: int,
                        scale=None, scale_q: Meta8 | None = None, out=None, stream=None):
    """Dequantize a matrix whose zero points (and optionally scales) are kept in
    8-bit form, in one pass (see include/hqq.h)."""
    if stream is not None:
        return _on(stream, packed, hqq_dequantize_meta, packed, zero_q, rows, cols, nbits, group,
                   scale, scale_q, out)
    import torch
    for t, nm in ((packed, "packed"), (scale, "scale"), (out, "out")):
        _check_tensor(t, nm)
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float16, device=packed.device)
    zc = zero_q._c()
    sc = scale_q._c() if scale_q is not None else None
    _check(_lib.hqq_dequantize_meta(_ptr(packed), ctypes.byref(zc), _ptr(scale),
                                    ctypes.byref(sc) if sc is not None else None,
                                    rows, cols, nbits, group, _ptr(out), _stream()))
    return out


def hqq_linear(X, q: QuantizedMatrix, out=None, status=None, stream=None):
    """Y = X W_hat^T for fp16 X [M, cols] and a quantized [rows, cols] matrix,
    with the dequantization fused into the tensor-core product (see
    include/hqq.h).  ``status`` is an optional int32 CUDA tensor of one element
    (cleared by the caller) that the kernel sets to 1 if an internal wait ran
    out."""
    if stream is not None:
        return _on(stream, X, hqq_linear, X, q, out, status)
    import torch
    if X.dtype != torch.float16 or X.dim() != 2 or X.shape[1] != q.cols:
        raise ValueError("X must be a float16 [M, cols] tensor")
    for t, nm in ((X, "X"), (q.packed, "packed"), (q.scale, "scale"), (q.zero, "zero"),
                  (out, "out"), (status, "status")):
        _check_tensor(t, nm)
    if out is None:
        out = torch.empty((X.shape[0], q.rows), dtype=torch.float16, device=X.device)
    _check(_lib.hqq_linear(_ptr(X), X.shape[0], _ptr(q.packed), _ptr(q.scale), _ptr(q.zero),
                           q.rows, q.cols, q.nbits, q.group, _ptr(out), _ptr(status),
                           _stream()))
    return out


def hqq_linear_meta(X, packed, zero_q: Meta8, rows: int, cols: int, nbits: int, group: int,
                    scale=None, scale_q: Meta8 | None = None, out=None, status=None,
                    stream=None):
    """hqq_linear for a matrix whose zero points (and optionally scales) are
    kept in 8-bit form; they are restored inside the kernel (see include/hqq.h)."""
    if stream is not None:
        return _on(stream, X, hqq_linear_meta, X, packed, zero_q, rows, cols, nbits, group, scale,
                   scale_q, out, status)
    import torch
    if X.dtype != torch.float16 or X.dim() != 2 or X.shape[1] != cols:
        raise ValueError("X must be a float16 [M, cols] tensor")
    for t, nm in ((X, "X"), (packed, "packed"), (scale, "scale"), (out, "out"),
                  (status, "status")):
        _check_tensor(t, nm)
    if out is None:
        out = torch.empty((X.shape[0], rows), dtype=torch.float16, device=X.device)
    zc = zero_q._c()
    sc = scale_q._c() if scale_q is not None else None
    _check(_lib.hqq_linear_meta(_ptr(X), X.shape[0], _ptr(packed), ctypes.byref(zc),
                                _ptr(scale), ctypes.byref(sc) if sc is not None else None,
                                rows, cols, nbits, group, _ptr(out), _ptr(status),
                                _stream()))
    return out


def hqq_lowrank(W, q: QuantizedMatrix, rank: int, omega, power_iters: int = 2, workspace=None,
                stream=None):
    """Rank-r residual B [rows, rank], A [rank, cols] (fp32) of the quantization
    error W - W_hat, with the r leading singular values (see include/hqq.h).
    ``omega`` is the fp32 [cols, sketch] Gaussian test matrix (sketch 16, 32 or
    64), drawn by the caller; the workspace is allocated here unless given."""
    if stream is not None:
        return _on(stream, W, hqq_lowrank, W, q, rank, omega, power_iters, workspace)
    import torch
    if W.dtype != torch.float16 or tuple(W.shape) != (q.rows, q.cols):
        raise ValueError("W must be the float16 [rows, cols] matrix that q quantizes")
    if omega.dtype != torch.float32 or omega.dim() != 2 or omega.shape[0] != q.cols:
        raise ValueError("omega must be a float32 [cols, sketch] tensor")
    for t, nm in ((W, "W"), (omega, "omega"), (workspace, "workspace")):
        _check_tensor(t, nm)
    sketch = omega.shape[1]
    need = _lib.hqq_lowrank_workspace_bytes(q.rows, q.cols, sketch)
    if need < 0:
        raise ValueError("sketch must be 16, 32 or 64")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=W.device)
    B = torch.empty((q.rows, rank), dtype=torch.float32, device=W.device)
    A = torch.empty((rank, q.cols), dtype=torch.float32, device=W.device)
    sigma = torch.empty(rank, dtype=torch.float32, device=W.device)
    _check(_lib.hqq_lowrank(_ptr(W), _ptr(q.packed), _ptr(q.scale), _ptr(q.zero), q.rows, q.cols,
                            q.nbits, q.group, rank, sketch, power_iters, _ptr(omega), _ptr(B),
                            _ptr(A), _ptr(sigma), _ptr(workspace), workspace.numel(),
                            _stream()))
    return B, A, sigma


_DTYPES = {}


def _dtype_code(dtype, name):
    """hqq_dtype of a torch dtype."""
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float16, bfloat16 or float32")
    return code


def _addr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dev):
    """A contiguous tensor on CUDA device dev (None passes)."""
    if t is not None and (t.get_device() != dev or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous tensor on cuda:{dev}")


def _run_on(dev, fn, *args):
    """fn(*args, stream) with CUDA device dev current, on its current stream."""
    import torch
    stream = torch.cuda.current_stream(dev)
    if torch.cuda.current_device() == dev:
        st = fn(*args, stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream.cuda_stream)
    if st != 0:
        raise HQQError(st)


def hqq_distill(logits, top_logits, top_index, temperature: float = 1.0, teacher_lse=None,
                weight=None, grad=False, loss=None, lse=None, stream=None):
    """Distillation loss of student ``logits`` [tokens, vocab] (fp16, bf16 or
    fp32; rows may be strided) against a teacher's stored entries
    ``top_logits`` / ``top_index`` [tokens, top_k] (index int32 or int64; an index
    outside the vocabulary is unused), and its gradient (see include/hqq.h).
    ``teacher_lse`` is the teacher's log-sum-exp over its whole vocabulary
    (without it the entries are normalised to sum 1), ``weight`` a factor per
    token (0: the token is skipped).  ``grad`` is False, True, or the tensor to
    write the gradient to, which may be ``logits`` itself.  Returns
    (loss [tokens], lse [tokens], gradient or None)."""
    if stream is not None:
        return _on(stream, logits, hqq_distill, logits, top_logits, top_index, temperature,
                   teacher_lse, weight, grad, loss, lse)
    import torch
    if logits.dim() != 2 or not logits.is_cuda or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a CUDA [tokens, vocab] tensor with adjacent columns")
    dt = _dtype_code(logits.dtype, "logits")
    tokens, vocab = logits.shape
    dev = logits.get_device()
    if top_logits.dim() != 2 or top_logits.shape != top_index.shape or \
            top_logits.shape[0] != tokens:
        raise ValueError("top_logits and top_index must be [tokens, top_k] tensors")
    if top_index.dtype not in (torch.int32, torch.int64):
        raise ValueError("top_index must be int32 or int64")
    _need(top_logits, "top_logits", dev)
    _need(top_index, "top_index", dev)
    for t, nm in ((teacher_lse, "teacher_lse"), (weight, "weight"), (loss, "loss"), (lse, "lse")):
        if t is not None:
            _need(t, nm, dev)
            if t.dtype != torch.float32 or t.numel() != tokens:
                raise ValueError(f"{nm} must be a float32 [tokens] tensor")
    if grad is True:
        grad = torch.empty_like(logits) if logits.is_contiguous() else \
            torch.empty((tokens, vocab), dtype=logits.dtype, device=logits.device)
    elif grad is False:
        grad = None
    elif grad.dtype != logits.dtype or grad.shape != logits.shape or \
            grad.get_device() != dev or (vocab > 1 and grad.stride(1) != 1):
        raise ValueError("grad must be like logits")
    if loss is None:
        loss = logits.new_empty(tokens, dtype=torch.float32)
    if lse is None:
        lse = torch.empty_like(loss)
    # (a single row may report any stride)
    rows = grows = vocab
    if tokens > 1:
        rows = logits.stride(0)
        grows = vocab if grad is None else grad.stride(0)
        if rows < vocab or grows < vocab:
            raise ValueError("rows of logits and grad must not overlap")
    _run_on(dev, _lib.hqq_distill, logits.data_ptr(), rows, dt, tokens, vocab,
            top_logits.data_ptr(), _dtype_code(top_logits.dtype, "top_logits"),
            top_index.data_ptr(), top_index.element_size(), top_logits.shape[1], temperature,
            _addr(teacher_lse), _addr(weight), loss.data_ptr(), lse.data_ptr(), _addr(grad), grows)
    return loss, lse, grad


@dataclass
class Adapters:
    """Low-rank adapters of one rank beside a quantized matrix: the pair of
    adapter a adds scaling[a] * B[a] A[a].  A 2-D pair (hqq_lowrank's B and A) is one adapter."""
    A: "torch.Tensor"          # fp16, bf16 or fp32 [count, rank, cols] (or [rank, cols])
    B: "torch.Tensor"          # the same type  [count, rows, rank] (or [rows, rank])
    scaling: "torch.Tensor | None" = None   # fp32 [count]; None: 1

    def _c(self, rows: int, cols: int, dev: int):
        A, B, scaling = self.A, self.B, self.scaling
        if A.dim() == 2:
            A = A.unsqueeze(0)
        if B.dim() == 2:
            B = B.unsqueeze(0)
        if A.dim() != 3 or B.dim() != 3:
            raise ValueError("adapters must be A [count, rank, cols] and B [count, rows, rank]")
        count, rank, ac = A.shape
        if B.shape != (count, rows, rank) or ac != cols:
            raise ValueError("adapters must be A [count, rank, cols] and B [count, rows, rank]")
        if A.dtype != B.dtype:
            raise ValueError("A and B must have the same type")
        a_stride = b_stride = 0
        if not (A.is_contiguous() and B.is_contiguous()):
            for t, nm in ((A, "A"), (B, "B")):
                if t.numel() and not t[0].is_contiguous():
                    raise ValueError(f"each adapter's {nm} must be a contiguous matrix")
                if count > 1 and t.stride(0) < t.shape[1] * t.shape[2]:
                    raise ValueError(f"the adapters of {nm} must not overlap")
            if count > 1:
                a_stride, b_stride = A.stride(0), B.stride(0)
        if A.get_device() != dev or B.get_device() != dev:
            raise ValueError(f"adapters must be on cuda:{dev}")
        s = None
        if scaling is not None:
            _need(scaling, "scaling", dev)
            if _dtype_code(scaling.dtype, "scaling") != 2 or scaling.numel() != count:
                raise ValueError("scaling must be a float32 [count] tensor")
            s = scaling.data_ptr()
        return _CAdapters(A.data_ptr(), B.data_ptr(), s, a_stride, b_stride, count, rank,
                          _dtype_code(A.dtype, "adapters"))


def _adapter_call(fn, lead, tail, x, q, adapters, index, zero_q, scale_q, M, backward, workspace,
                  tensors):
    """What both adapter calls check and marshal: fn(*lead, matrix, adapters, index, *tail,
    workspace, its bytes, stream)."""
    import torch
    if index is not None and (index.dtype != torch.int32 or index.numel() != M):
        raise ValueError("index must be an int32 [M] tensor")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    zero = q.zero if zero_q is None else None
    scale = q.scale if scale_q is None else None
    for t, nm in ((q.packed, "packed"), (index, "index"), (workspace, "workspace"),
                  (zero, "zero"), (scale, "scale"), *tensors):
        _need(t, nm, dev)
    ca, rank, count = None, 0, 0
    if adapters is not None:
        ca = adapters._c(q.rows, q.cols, dev)
        rank, count = ca.rank, ca.count
    for m in (zero_q, scale_q):
        if m is not None:
            for t in (m.codes, m.scale, m.zero):
                _need(t, "8-bit meta data", dev)
    need = _lib.hqq_linear_adapters_workspace_bytes(M, q.rows, q.cols, rank, count, backward)
    if need < 0:
        raise HQQError(2 if ca is None or (0 < rank <= 512 and 0 < count <= 65535) else 4)
    if workspace is None and need:
        workspace = x.new_empty(need, dtype=torch.uint8)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    byref = ctypes.byref
    _run_on(dev, fn, *lead, M, q.packed.data_ptr(), _addr(scale), _addr(zero),
            None if zero_q is None else byref(zero_q._c()),
            None if scale_q is None else byref(scale_q._c()), q.rows, q.cols, q.nbits, q.group,
            None if ca is None else byref(ca), _addr(index), *tail, _addr(workspace), nbytes)


def hqq_linear_adapters(X, q: QuantizedMatrix, adapters: Adapters, index=None, out=None,
                        status=None, workspace=None, zero_q: Meta8 | None = None,
                        scale_q: Meta8 | None = None, stream=None):
    """hqq_linear plus each token's adapter (see include/hqq.h): ``index`` is an
    int32 [M] tensor (negative or past the last: none), or None for adapter 0
    everywhere.  ``zero_q`` / ``scale_q`` replace q's zero / scale by their 8-bit
    form.  The workspace is allocated here unless given."""
    if stream is not None:
        return _on(stream, X, hqq_linear_adapters, X, q, adapters, index, out, status, workspace,
                   zero_q, scale_q)
    import torch
    if X.dtype != torch.float16 or X.dim() != 2 or X.shape[1] != q.cols:
        raise ValueError("X must be a float16 [M, cols] tensor")
    M = X.shape[0]
    if out is None:
        out = X.new_empty((M, q.rows))
    elif out.dtype != torch.float16 or out.numel() != M * q.rows:
        raise ValueError("out must be a float16 [M, rows] tensor")
    _adapter_call(_lib.hqq_linear_adapters, (X.data_ptr(),), (out.data_ptr(), _addr(status)), X, q,
                  adapters, index, zero_q, scale_q, M, 0, workspace,
                  ((X, "X"), (out, "out"), (status, "status")))
    return out


def hqq_linear_adapters_backward(dY, X, q: QuantizedMatrix, adapters: Adapters | None = None,
                                 index=None, need_dX: bool = True, need_factors: bool = True,
                                 dX=None, dA=None, dB=None, status=None, workspace=None,
                                 zero_q: Meta8 | None = None, scale_q: Meta8 | None = None,
                                 stream=None):
    """Gradients (dX, dA, dB) of hqq_linear_adapters for the output's gradient
    ``dY`` [M, rows] (see include/hqq.h): dX fp16 [M, cols], dA fp32 [count, rank,
    cols], dB fp32 [count, rows, rank].  Without adapters (X may then be None),
    or for what need_dX / need_factors leaves out, None is returned in its place."""
    if stream is not None:
        return _on(stream, dY, hqq_linear_adapters_backward, dY, X, q, adapters, index, need_dX,
                   need_factors, dX, dA, dB, status, workspace, zero_q, scale_q)
    import torch
    if dY.dtype != torch.float16 or dY.dim() != 2 or dY.shape[1] != q.rows:
        raise ValueError("dY must be a float16 [M, rows] tensor")
    M = dY.shape[0]
    need_factors = need_factors and adapters is not None
    if adapters is None and (index is not None or dA is not None or dB is not None):
        raise ValueError("index, dA and dB need adapters")
    if not need_factors:
        X = None
    elif X is None or X.dtype != torch.float16 or tuple(X.shape) != (M, q.cols):
        raise ValueError("X must be a float16 [M, cols] tensor")
    if not need_dX:
        dX = None
    elif dX is None:
        dX = dY.new_empty((M, q.cols))
    elif dX.dtype != torch.float16 or dX.numel() != M * q.cols:
        raise ValueError("dX must be a float16 [M, cols] tensor")
    if need_factors:
        count = adapters.A.shape[0] if adapters.A.dim() == 3 else 1
        rank = adapters.A.shape[-2]
        if dA is None:
            dA = dY.new_empty((count, rank, q.cols), dtype=torch.float32)
        if dB is None:
            dB = dY.new_empty((count, q.rows, rank), dtype=torch.float32)
        if dA.dtype != torch.float32 or dA.numel() != count * rank * q.cols or \
                dB.dtype != torch.float32 or dB.numel() != count * rank * q.rows:
            raise ValueError("dA and dB must be float32 [count, rank, cols] and "
                             "[count, rows, rank] tensors")
    else:
        dA = dB = None
    _adapter_call(_lib.hqq_linear_adapters_backward, (dY.data_ptr(), _addr(X)),
                  (_addr(dX), _addr(dA), _addr(dB), _addr(status)), dY, q, adapters, index, zero_q,
                  scale_q, M, 1, workspace,
                  ((dY, "dY"), (X, "X"), (dX, "dX"), (dA, "dA"), (dB, "dB"), (status, "status")))
    return dX, dA, dB
