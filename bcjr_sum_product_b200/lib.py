"""Thin ctypes binding of ``libbcjr.so`` (include/bcjr.h).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  torch is used for device memory and streams.  There
is no CPU fallback: if the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbcjr.so")

BCJR_OK = 0
BCJR_ERR_INVALID_ARG = 1
BCJR_ERR_UNSUPPORTED = 2
BCJR_ERR_CUDA = 3
BCJR_ERR_TIMEOUT = 4
BCJR_ERR_NUMERIC = 5

EXPORTS = ("bcjr_soft_codeword", "bcjr_vjp", "viterbi_decode", "bcjr_posterior_argmax",
           "bcjr_fp8_quantise", "bcjr_fp8_matmul", "bcjr_orthogonalise", "bcjr_muon_step",
           "bcjr_get_device_error", "bcjr_launch_count", "bcjr_strerror", "bcjr_version")


class BcjrError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load the library (building it in-tree first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            from . import build as _build
            if _build.needs_build():
                _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"libbcjr.so not found at {path}")
            lib = ctypes.CDLL(path)
            P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
            lib.bcjr_soft_codeword.argtypes = [P, i64, i64, i32, i32, i32, P, f32, P, P, P]
            lib.bcjr_vjp.argtypes = [P, i64, i64, i32, i32, i32, P, f32, P, P, P, P, P]
            lib.viterbi_decode.argtypes = [P, i64, i64, i32, i32, i32, P, P, P, P]
            lib.bcjr_posterior_argmax.argtypes = [P, i64, i64, i32, i32, i32, P, f32, P, P]
            lib.bcjr_qat_step.argtypes = [P, P, i64, i64, i32, i32, i32, P, f32, f32, f32, P, P, P, P, P]
            lib.bcjr_fp8_quantise.argtypes = [P, i32, i64, i64, i64, P, i64, i32, i32, P, i64, P, i64, P, i64, P,
                                              i64, P]
            lib.bcjr_fp8_matmul.argtypes = [P, i32, i64, P, i64, i32, P, i32, i64, P, i64, i32, i64, i64, i64, f32, P,
                                            i32, i64, P]
            lib.bcjr_orthogonalise.argtypes = [P, i32, i64, i64, i64, i64, i64, i32, P, f32, P, i32, i64, i64, P]
            lib.bcjr_muon_step.argtypes = [P, i64, P, i32, i64, P, i64, i64, i64, f32, f32, i32, f32, f32, i32, P, f32,
                                           P]
            lib.bcjr_get_device_error.argtypes = [P]
            lib.bcjr_strerror.argtypes = [i32]
            lib.bcjr_strerror.restype = ctypes.c_char_p
            lib.bcjr_version.argtypes = []
            lib.bcjr_version.restype = ctypes.c_char_p
            lib.bcjr_launch_count.argtypes = []
            lib.bcjr_launch_count.restype = ctypes.c_uint64
            for name in ("bcjr_soft_codeword", "bcjr_vjp", "viterbi_decode", "bcjr_posterior_argmax",
                         "bcjr_qat_step", "bcjr_fp8_quantise", "bcjr_fp8_matmul", "bcjr_orthogonalise",
                         "bcjr_muon_step", "bcjr_get_device_error"):
                getattr(lib, name).restype = ctypes.c_int
            _lib = lib
    return _lib


def strerror(status: int) -> str:
    return load().bcjr_strerror(int(status)).decode()


def launch_count() -> int:
    """bcjr_launch_count: kernels the library has launched in this process."""
    return int(load().bcjr_launch_count())


def version() -> str:
    return load().bcjr_version().decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev(t: torch.Tensor, name: str, dtype=torch.float32) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _check(rc: int, where: str):
    if rc != BCJR_OK:
        raise BcjrError(rc, where)


def soft_codeword(w: torch.Tensor, codebook: torch.Tensor, L: int, k: int, V: int, T: float,
                  out_soft: Optional[torch.Tensor] = None, out_logZ: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """bcjr_soft_codeword: soft codeword [n_seq, len] and natural-log logZ [n_seq]."""
    _dev(w, "w"); _dev(codebook, "codebook")
    n_seq, seq_len = w.shape
    if out_soft is None:
        out_soft = torch.empty_like(w)
    if out_logZ is None:
        out_logZ = torch.empty(n_seq, device=w.device, dtype=torch.float32)
    rc = load().bcjr_soft_codeword(_ptr(w), n_seq, seq_len, L, k, V, _ptr(codebook), float(T), _ptr(out_soft),
                                   _ptr(out_logZ), _stream(stream))
    _check(rc, "bcjr_soft_codeword")
    return out_soft, out_logZ


def vjp(w: torch.Tensor, codebook: torch.Tensor, L: int, k: int, V: int, T: float, grad_soft: torch.Tensor,
        grad_logZ: Optional[torch.Tensor] = None, grad_w: Optional[torch.Tensor] = None,
        grad_codebook: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """bcjr_vjp: (dl/dw [n_seq, len], dl/dcodebook [2^L(, V)])."""
    _dev(w, "w"); _dev(codebook, "codebook"); _dev(grad_soft, "grad_soft")
    if grad_logZ is not None:
        _dev(grad_logZ, "grad_logZ")
    n_seq, seq_len = w.shape
    if grad_w is None:
        grad_w = torch.empty_like(w)
    if grad_codebook is None:
        grad_codebook = torch.empty_like(codebook)
    rc = load().bcjr_vjp(_ptr(w), n_seq, seq_len, L, k, V, _ptr(codebook), float(T), _ptr(grad_soft),
                         _ptr(grad_logZ), _ptr(grad_w), _ptr(grad_codebook), _stream(stream))
    _check(rc, "bcjr_vjp")
    return grad_w, grad_codebook


def qat_step(w: torch.Tensor, w_target: torch.Tensor, codebook: torch.Tensor, L: int, k: int, V: int, T: float,
             lr_w: float, lr_c: float = 0.0, out_soft: Optional[torch.Tensor] = None,
             out_loss: Optional[torch.Tensor] = None, grad_w: Optional[torch.Tensor] = None,
             grad_codebook: Optional[torch.Tensor] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """bcjr_qat_step: one self-reconstruction QAT step; updates ``w`` (and the
    codebook when ``lr_c`` != 0) in place and returns (w_hat, loss per sequence,
    dl/dw, dl/dcodebook), all taken before the update."""
    _dev(w, "w"); _dev(w_target, "w_target"); _dev(codebook, "codebook")
    n_seq, seq_len = w.shape
    if tuple(w_target.shape) != (n_seq, seq_len):
        raise ValueError("w_target must have the shape of w")
    if out_soft is None:
        out_soft = torch.empty_like(w)
    if out_loss is None:
        out_loss = torch.empty(n_seq, device=w.device, dtype=torch.float32)
    if grad_w is None:
        grad_w = torch.empty_like(w)
    if grad_codebook is None:
        grad_codebook = torch.empty_like(codebook)
    rc = load().bcjr_qat_step(_ptr(w), _ptr(w_target), n_seq, seq_len, L, k, V, _ptr(codebook), float(T),
                              float(lr_w), float(lr_c), _ptr(out_soft), _ptr(out_loss), _ptr(grad_w),
                              _ptr(grad_codebook), _stream(stream))
    _check(rc, "bcjr_qat_step")
    return out_soft, out_loss, grad_w, grad_codebook


def viterbi_decode(w: torch.Tensor, codebook: torch.Tensor, L: int, k: int, V: int,
                   out_states: Optional[torch.Tensor] = None, out_cost: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """viterbi_decode: (states [n_seq, n] int32, cost [n_seq] fp32)."""
    _dev(w, "w"); _dev(codebook, "codebook")
    n_seq, seq_len = w.shape
    n = seq_len // V
    if out_states is None:
        out_states = torch.empty((n_seq, n), device=w.device, dtype=torch.int32)
    if out_cost is None:
        out_cost = torch.empty(n_seq, device=w.device, dtype=torch.float32)
    rc = load().viterbi_decode(_ptr(w), n_seq, seq_len, L, k, V, _ptr(codebook), _ptr(out_states),
                               _ptr(out_cost), _stream(stream))
    _check(rc, "viterbi_decode")
    return out_states, out_cost


def posterior_argmax(w: torch.Tensor, codebook: torch.Tensor, L: int, k: int, V: int, T: float,
                     out_argmax: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bcjr_posterior_argmax: argmax_s p_t(s) per step, [n_seq, n] int32."""
    _dev(w, "w"); _dev(codebook, "codebook")
    n_seq, seq_len = w.shape
    n = seq_len // V
    if out_argmax is None:
        out_argmax = torch.empty((n_seq, n), device=w.device, dtype=torch.int32)
    rc = load().bcjr_posterior_argmax(_ptr(w), n_seq, seq_len, L, k, V, _ptr(codebook), float(T),
                                      _ptr(out_argmax), _stream(stream))
    _check(rc, "bcjr_posterior_argmax")
    return out_argmax


def get_device_error(stream=None) -> int:
    return int(load().bcjr_get_device_error(_stream(stream)))


def soft_codeword_noalloc(w: torch.Tensor, codebook: torch.Tensor, L: int, k: int, V: int, T: float,
                          out_soft: Optional[torch.Tensor] = None, out_logZ: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """bcjr_soft_codeword_noalloc: as soft_codeword, but the library allocates
    nothing (its scratch is a fixed 64 MiB device array shared by all calls on a
    device; calls that overlap on the GPU race on it).  For callers that may not
    allocate device memory; the output tensors are still the caller's."""
    _dev(w, "w"); _dev(codebook, "codebook")
    n_seq, seq_len = w.shape
    if out_soft is None:
        out_soft = torch.empty_like(w)
    if out_logZ is None:
        out_logZ = torch.empty(n_seq, device=w.device, dtype=torch.float32)
    fn = load().bcjr_soft_codeword_noalloc
    P = ctypes.c_void_p
    fn.argtypes = [P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, P, ctypes.c_float,
                   P, P, P]
    fn.restype = ctypes.c_int
    rc = fn(_ptr(w), n_seq, seq_len, L, k, V, _ptr(codebook), float(T), _ptr(out_soft), _ptr(out_logZ),
            _stream(stream))
    _check(rc, "bcjr_soft_codeword_noalloc")
    return out_soft, out_logZ


# ---------------------------------------------------------------- layer-wise QAT

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3, torch.float8_e5m2: 4}
_WIDE = (torch.float32, torch.float16, torch.bfloat16)
_CODES = (torch.float8_e4m3fn, torch.float8_e5m2)
_SCALES = (torch.float8_e8m0fnu,)
_SCALE_NAMES = {"a": "scale_a", "b": "scale_b"}
_BLOCK = 128
_empty = torch.empty_strided
#: Coefficients of Muon's Newton-Schulz step (the default of orthogonalise and muon_step).
MUON_COEFFS = (3.4445, -4.7750, 2.0315)


def _matrix(t: torch.Tensor, name: str, dtypes, ndim: int = 2, device=None) -> torch.Tensor:
    """A CUDA matrix whose rows are contiguous (any row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}")
    stride = t.stride()
    if len(stride) != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if not t.is_contiguous():
        shape = t.shape
        if stride[-1] != 1 and shape[-1] > 1:
            raise ValueError(f"the last dimension of {name} must be contiguous")
        if stride[-2] < shape[-1] and shape[-2] > 1:
            raise ValueError(f"the rows of {name} must not overlap")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t


def _ld(t: torch.Tensor) -> int:
    """Row stride in elements (for a single row, its length)."""
    return t.stride(-2) if t.shape[-2] > 1 else t.shape[-1]


def _overlap(p: torch.Tensor, q: torch.Tensor) -> bool:
    """Whether two matrices share memory; rows that lie between the other's rows do not."""
    (rows_p, cols_p), (rows_q, cols_q) = p.shape, q.shape
    if not (rows_p and cols_p and rows_q and cols_q):
        return False
    at_p, size_p = p.data_ptr(), p.element_size()
    at_q, size_q = q.data_ptr(), q.element_size()
    ld_p, ld_q, row_p, row_q = _ld(p) * size_p, _ld(q) * size_q, cols_p * size_p, cols_q * size_q
    if at_p + (rows_p - 1) * ld_p + row_p <= at_q or at_q + (rows_q - 1) * ld_q + row_q <= at_p:
        return False
    # for each row of p the last row of q that starts before its end
    start_p = at_p + ld_p * torch.arange(rows_p)
    start_q = at_q + ld_q * torch.arange(rows_q)
    last = torch.searchsorted(start_q, start_p + row_p) - 1
    return bool(((last >= 0) & (start_q[last.clamp_min(0)] + row_q > start_p)).any())


def _no_gradient(where: str, *tensors):
    """These operators have no derivative: a result that silently lacks one is refused."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise RuntimeError(f"{where} has no derivative: detach its inputs, or call it under torch.no_grad()")


def _changed(*tensors):
    """Tells autograd that the tensors were written."""
    torch.autograd.graph.increment_version([t for t in tensors if not t.is_inference()])


def _apart(named, out: torch.Tensor, name: str):
    for other, t in named:
        if _overlap(out, t):
            raise ValueError(f"{name} and {other} must not share memory")


def _raw_stream(index: int) -> int:
    """Handle of a device's current stream."""
    return torch._C._cuda_getCurrentRawStream(index)


def _call(device: torch.device, stream, fn, *args):
    """fn(*args, stream handle) with the tensors' device current, on the given
    stream or that device's current one (allocations belong to it too)."""
    if stream is None and device.index == torch.cuda.current_device():
        return fn(*args, _raw_stream(device.index))
    with torch.cuda.device(device):
        if stream is None:
            return fn(*args, torch.cuda.current_stream().cuda_stream)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
        if stream.device != device:
            raise ValueError(f"stream must be on {device}")
        with torch.cuda.stream(stream):
            return fn(*args, stream.cuda_stream)


def _codes_room(rows: int, cols: int, block_rows: int, dtype, device):
    """Codes [rows, cols] and scales in rows of a multiple of 16 bytes; and pointer and row stride of each for the call."""
    ld, blocks = (cols + 15) // 16 * 16, (cols + 127) // 128
    ld_s = (blocks + 15) // 16 * 16
    q = _empty((rows, cols), (ld, 1), dtype=dtype, device=device)
    s = _empty((rows if block_rows == 1 else (rows + 127) // 128, blocks), (ld_s, 1), dtype=torch.float8_e8m0fnu, device=device)
    return (q, s), (q.data_ptr(), ld, s.data_ptr(), ld_s)


_NO_CODES = ((), (None, 0, None, 0))


def fp8_quantise(x: torch.Tensor, block_rows: int = 1, dtype: torch.dtype = torch.float8_e4m3fn,
                 minus: Optional[torch.Tensor] = None, layout: str = "rows", stream=None) -> Tuple[torch.Tensor, ...]:
    """bcjr_fp8_quantise: 8-bit codes of a matrix ``x`` (fp32, fp16, bf16; ``x - minus``
    with an fp32 ``minus``) and their power-of-two scales, one for each 128 values of
    a row (``block_rows`` 1) or for each 128 x 128 block (``block_rows`` 128).

    ``layout`` "rows" returns (codes [rows, cols], scales [ceil(rows / block_rows),
    ceil(cols / 128)] float8_e8m0fnu); "cols" the same of the transpose of x
    (codes [cols, rows], blocks down the columns of x); "both" all four, from one
    pass over x.  The rows of the codes start at multiples of 16 bytes, as
    fp8_matmul takes them.  No derivative: an input that requires one is refused outside
    torch.no_grad (so it is by fp8_matmul and orthogonalise)."""
    _matrix(x, "x", _WIDE)
    if block_rows not in (1, _BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    if dtype not in _CODES:
        raise TypeError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2")
    if layout not in ("rows", "cols", "both"):
        raise ValueError('layout must be "rows", "cols" or "both"')
    if minus is not None:
        _matrix(minus, "minus", (torch.float32,), device=x.device)
        if minus.shape != x.shape:
            raise ValueError("minus must have the shape of x")
    _no_gradient("fp8_quantise", x, minus)
    return _call(x.device, stream, _fp8_quantise, x, block_rows, dtype, minus, layout)


def _fp8_quantise(x, block_rows, dtype, minus, layout, st):
    rows, cols = x.shape
    device = x.device
    out, room = _codes_room(rows, cols, block_rows, dtype, device) if layout != "cols" else _NO_CODES
    out_t, room_t = _codes_room(cols, rows, block_rows, dtype, device) if layout != "rows" else _NO_CODES
    minus_p, ld_minus = (None, 0) if minus is None else (minus.data_ptr(), _ld(minus))
    rc = load().bcjr_fp8_quantise(x.data_ptr(), _TYPES[x.dtype], rows, cols, _ld(x), minus_p, ld_minus, _TYPES[dtype],
                                  block_rows, *room, *room_t, st)
    if rc:
        _check(rc, "bcjr_fp8_quantise")
    return out + out_t


def _scaled(q: torch.Tensor, scale: torch.Tensor, name: str, device):
    """Checks codes and their scales; returns the codes' shape and the call's
    pointer, type and row stride of the codes, pointer and row stride of the
    scales, and the rows that share a scale."""
    _matrix(q, name, _CODES, device=device)
    _matrix(scale, _SCALE_NAMES[name], _SCALES, device=device)
    rows, cols = shape = q.shape
    have = scale.shape
    blocks = (cols + _BLOCK - 1) // _BLOCK
    block_rows = 1 if have[0] == rows else _BLOCK
    if have[1] != blocks or have[0] != (rows + block_rows - 1) // block_rows:
        raise ValueError(f"scale_{name} must be [{rows}, {blocks}] or [{-(-rows // _BLOCK)}, {blocks}]")
    ptr, ld = q.data_ptr(), q.stride(0) if rows > 1 else (cols + 15) // 16 * 16
    if (ld % 16 or ptr % 16) and rows and cols:
        raise ValueError(f"the rows of {name} must start at multiples of 16 bytes")
    return shape, (ptr, _TYPES[q.dtype], ld, scale.data_ptr(), scale.stride(0) if have[0] > 1 else blocks, block_rows)


def fp8_matmul(a: torch.Tensor, scale_a: torch.Tensor, b: torch.Tensor, scale_b: torch.Tensor, alpha: float = 1.0,
               out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """bcjr_fp8_matmul: alpha (a scale_a) (b scale_b)^T, [M, N], from 8-bit codes a [M, K]
    and b [N, K] (e4m3 or e5m2 each) with one scale for each 128 values of K and
    each row or 128 rows, as fp8_quantise gives them.  Sums are in fp32, the
    result (fp32, fp16 or bf16; ``out``, if given, with any row stride and apart from
    the operands) is rounded once."""
    (M, K), args_a = _scaled(a, scale_a, "a", None)
    device = a.device
    (N, Kb), args_b = _scaled(b, scale_b, "b", device)
    if K != Kb:
        raise ValueError("a and b must have the same number of columns")
    _no_gradient("fp8_matmul", a, b, out)
    if out is None:
        if out_dtype not in _WIDE:
            raise TypeError("out_dtype must be torch.float32, torch.float16 or torch.bfloat16")
    else:
        _matrix(out, "out", _WIDE, device=device)
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out must be [{M}, {N}]")
        _apart((("a", a), ("scale_a", scale_a), ("b", b), ("scale_b", scale_b)), out, "out")
    return _call(device, stream, _fp8_matmul, args_a, args_b, M, N, K, alpha, out_dtype, out, device)


def _fp8_matmul(args_a, args_b, M, N, K, alpha, out_dtype, out, device, st):
    if out is None:
        out, ld = _empty((M, N), (N, 1), dtype=out_dtype, device=device), N
    else:
        out_dtype, ld = out.dtype, _ld(out)
        _changed(out)
    rc = load().bcjr_fp8_matmul(*args_a, *args_b, M, N, K, float(alpha), out.data_ptr(), _TYPES[out_dtype], ld, st)
    _check(rc, "bcjr_fp8_matmul")
    return out


def _steps(steps) -> int:
    """A whole number of steps; what does not fit 32 bits as the limit that the library refuses."""
    if steps != steps or int(steps) != steps:
        raise ValueError("steps must be a whole number")
    return max(-1, min(int(steps), 1 << 16))


def _coeffs(coeffs, steps: int):
    """(a, b, c) for every step, or one triple for each, as a C array; None for the default."""
    if coeffs is None:
        return None
    flat = [float(v) for t in coeffs for v in (t if isinstance(t, (tuple, list)) else (t,))]
    if len(flat) == 3:
        flat = flat * max(steps, 1)
    if len(flat) != 3 * max(steps, 1):
        raise ValueError("coeffs must be (a, b, c) or one (a, b, c) for each step")
    return (ctypes.c_float * len(flat))(*flat)


def orthogonalise(g: torch.Tensor, steps: int = 5, coeffs: Optional[Sequence] = None, eps: float = 1e-7,
                  out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """bcjr_orthogonalise: Newton-Schulz orthogonalisation of a matrix or a batch of
    matrices ``g`` ([rows, cols] or [batch, rows, cols]; fp32, fp16, bf16) after
    division by its Frobenius norm + eps; bf16 or fp16 of the shape of g.
    Products sum in fp32.  With the default steps a bf16 result is within about 1e-3 (at
    most 2e-3) of the exact iteration in the 2-norm before it is rounded, an fp16 one
    (three times the work) within 1e-4 if g has many directions, up to 1.1e-3 if it has
    few.  ``coeffs`` is (a, b, c), or one such triple for each step; the default is
    Muon's."""
    if not isinstance(g, torch.Tensor) or g.dim() not in (2, 3):
        raise ValueError("g must be a matrix or a batch of matrices")
    _matrix(g, "g", _WIDE, ndim=g.dim())
    if out_dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float16")
    _no_gradient("orthogonalise", g)
    steps = _steps(steps)
    return _call(g.device, stream, _orthogonalise, g, steps, _coeffs(coeffs, steps), eps, out_dtype)


def _orthogonalise(g, steps, coeffs, eps, out_dtype, st):
    rows, cols = g.shape[-2:]
    out = torch.empty(g.shape, dtype=out_dtype, device=g.device)
    batch, stride = (g.shape[0], g.stride(0)) if g.dim() == 3 else (1, 0)
    rc = load().bcjr_orthogonalise(g.data_ptr(), _TYPES[g.dtype], batch, rows, cols, _ld(g), stride, steps, coeffs, float(eps),
                                   out.data_ptr(), _TYPES[out_dtype], cols, rows * cols, st)
    _check(rc, "bcjr_orthogonalise")
    return out


def muon_step(w: torch.Tensor, grad: torch.Tensor, momentum: torch.Tensor, lr: float, mu: float = 0.95,
              nesterov: bool = True, weight_decay: float = 0.0, scale: Optional[float] = None, steps: int = 5,
              coeffs: Optional[Sequence] = None, eps: float = 1e-7, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """bcjr_muon_step: one Muon step on a weight matrix; updates ``w`` and ``momentum``
    (fp32) in place from ``grad`` (fp32, fp16, bf16) and returns them:
    momentum = mu momentum + grad; u = grad + mu momentum (or momentum without
    nesterov); w = (1 - lr weight_decay) w - lr scale orthogonalise(u), the last within
    about 1e-3 in the 2-norm.
    ``scale`` defaults to sqrt(max(1, rows / cols)).  The three must not share memory.
    An optimizer's step: ``w`` may require a gradient, none is recorded."""
    _matrix(w, "w", (torch.float32,))
    _matrix(grad, "grad", _WIDE, device=w.device)
    _matrix(momentum, "momentum", (torch.float32,), device=w.device)
    if grad.shape != w.shape or momentum.shape != w.shape:
        raise ValueError("grad and momentum must have the shape of w")
    _apart((("momentum", momentum), ("grad", grad)), w, "w")
    _apart((("grad", grad),), momentum, "momentum")
    rows, cols = w.shape
    if scale is None:
        scale = math.sqrt(max(1.0, rows / cols)) if cols else 1.0
    steps = _steps(steps)
    return _call(w.device, stream, _muon_step, w, grad, momentum, lr, mu, int(bool(nesterov)), weight_decay, scale,
                 steps, _coeffs(coeffs, steps), eps)


def _muon_step(w, grad, momentum, lr, mu, nesterov, weight_decay, scale, steps, coeffs, eps, st):
    rows, cols = w.shape
    rc = load().bcjr_muon_step(w.data_ptr(), _ld(w), grad.data_ptr(), _TYPES[grad.dtype], _ld(grad), momentum.data_ptr(),
                               _ld(momentum), rows, cols, float(lr), float(mu), nesterov, float(weight_decay), float(scale), steps,
                               coeffs, float(eps), st)
    _check(rc, "bcjr_muon_step")
    _changed(w, momentum)
    return w, momentum
