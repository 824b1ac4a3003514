"""Python binding of libq8gemv, the GB300 Q8_0 block-quantized GEMV library.

Argument marshalling only: every step of the product runs in the library's CUDA kernels (device entry points) or its
C++ host code (repack, quantize).  PyTorch supplies device memory and streams: a call with ``stream=`` runs there, what
it allocates is allocated there, and the caller orders its inputs' writes before it.  The names follow the C ABI in
``include/q8_gemv.h``:

* :func:`gemv` -- ``q8_gemv`` / ``q8_gemv_ex``: y[r, n] = sum_b s[b, n] sum_i x[r, 32b+i] q[32b+i, n]
  ("from_q8.rs", module doc), bf16 x [m, K], int8 q [K, Np], fp32 s [K/32, Np] -> fp32 y [m, Np];
* :func:`gemv_argmax` -- ``q8_gemv_argmax``: the product and the first-maximum arg-max that ends a decode step;
* :func:`quantize_act` -- ``q8_quantize_act``: the quantized form of an activation (int8 values and an fp32 scale per
  32, "plan.rs" ``QBLOCK``); every product function takes the :class:`QuantAct` it returns in place of bf16 x
  (``Q8_FLAG_Q8_ACT``, tiled weights);
* :class:`KVCache`, :func:`kv_slots`, :func:`rope_table`, :func:`rope_append`, :func:`attn_decode`,
  :func:`attn_prefill` -- what lies between the q/k/v products and the output projection: a paged key-value cache
  (bf16 or Q8_0), its block tables and slots, the append with norms and rotation, and the attention over it;
* :class:`Weight4`, :func:`gemv4`, :func:`gemv4_parts`, :func:`gemv4_glu`, :func:`gemv4_residual_norm` -- the products
  over weights of 4 bits with a scale (and a zero point) for each group of 32, 64 or 128 rows; :func:`repack4` makes them
  from checkpoint blocks;
* :func:`choose` -- ``q8_choose``: penalties for repeated tokens, biases, temperature and grammar masks on the logits, and
  the token chosen;
* :func:`repack` -- ``q8_repack``: 36-byte checkpoint blocks -> (q, s) on the host;
* :func:`quantize` -- ``q8_quantize``: the Q8_0 rule of "from_q8.rs" ``quantize`` on the host.

The library must have been built (``python -m q8_block_quantized_gemv_gb300.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

from .build import LIB as _LIB_PATH

Q8_BLOCK = 32
MAX_ROWS = 16
MAX_CHUNK = 512  # rows one call over tiled weights takes
VARIANTS = {"auto": 0, "simt": 1, "mma": 2, "tma": 3}

_STATUS = {0: "Q8_OK", 1: "Q8_ERR_ARG", 2: "Q8_ERR_SHAPE", 3: "Q8_ERR_ALIGN", 4: "Q8_ERR_NOT_Q8_0", 5: "Q8_ERR_CUDA"}

# Every symbol include/q8_gemv.h declares, with its ctypes signature.
_P = ctypes.c_void_p
_I = ctypes.c_int
SIGNATURES = {
    "q8_padded_n": (_I, [_I]),
    "q8_gemv": (_I, [_P, _P, _P, _P, _I, _I, _I, _P]),
    "q8_gemv_ex": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_uint, _P]),
    "q8_gemv_argmax": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "q8_gemv_argmax_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, ctypes.c_uint, _P]),
    "q8_tiled_n": (_I, [_I]),
    "q8_tile": (_I, [_P, _P, _I, _I, _P, _P]),
    "q8_tile_device": (_I, [_P, _P, _I, _I, _P, _P, _P]),
    "q8_repack": (_I, [_P, _I, _I, _P, _P]),
    "q8_quantize": (_I, [_P, _I, _I, _P, _P]),
    "q8_status_string": (ctypes.c_char_p, [_I]),
    "q8_last_cuda_error": (_I, []),
    "q8_version": (_I, []),
    "q8_device_fault": (_I, [_P, _I]),
    "q8_gemv_parts": (_I, [_P, _P, _I, _I, _I, ctypes.c_uint, _P]),
    "q8_gemv_glu": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, ctypes.c_uint, _P]),
    "q8_gemv_residual_norm": (_I, [_P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _I, _I, _I, ctypes.c_uint, _P]),
    "q8_act_bytes": (ctypes.c_int64, [_I, _I]),
    "q8_repack_f16": (_I, [_P, _I, _I, _P, _P]),
    "q8_gemv_glu_ex": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, ctypes.c_uint, _P]),
    "q8_gemv_residual_norm_ex": (_I, [_P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P, _I, _I, _I, ctypes.c_uint, _P]),
    "q8_quantize_act": (_I, [_P, _P, _I, _I, _P]),
    "q8_gemv_residual_norm_noalloc": (_I, [_P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _I, _I, _I, ctypes.c_uint,
                                          _P]),
    "q8_plan_launches": (_I, [_I, _I, _P, _I, ctypes.c_uint]),
    "q8_plan_glu_launches": (_I, [_I, _I, _I, ctypes.c_uint]),
    "q8_set_tuning": (_I, [_I, _I]),
    "q8_get_tuning": (_I, [_I]),
    "q8_kv_slots": (_I, [_P, _P, _I, _I, _P, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "q8_rope_append": (_I, [_P, _I, _P, _I, _P, _I, _P, _P, ctypes.c_float, _P, _I, _I, _P, _P, _P, _I, _P, _I, _I,
                            ctypes.c_uint, _P]),
    "q8_attn_workspace_bytes": (ctypes.c_int64, []),
    "q8_attn_decode": (_I, [_P, _I, _P, _P, _I, _I, _P, _P, _I, _I, _I, ctypes.c_float, _I, _I, _P, _P]),
    "q8_attn_prefill": (_I, [_P, _I, _P, _P, _I, _I, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _I, _I, _P, _P]),
    "q8_w4_bytes": (ctypes.c_int64, [_I, _I, _I, ctypes.c_uint]),
    "q8_w4_tile": (_I, [_P, _P, _P, _I, _I, _I, ctypes.c_uint, _P]),
    "q8_w4_tile_device": (_I, [_P, _P, _P, _I, _I, _I, ctypes.c_uint, _P, _P]),
    "q8_w4_repack": (_I, [_P, _I, _I, _P, _P]),
    "q8_gemv4": (_I, [_P, _P, _P, _I, _I, ctypes.c_uint, _P]),
    "q8_gemv4_parts": (_I, [_P, _P, _P, _I, _I, _I, ctypes.c_uint, _P]),
    "q8_gemv4_glu": (_I, [_P, _P, _P, _P, _P, _I, _I, ctypes.c_uint, _P]),
    "q8_gemv4_residual_norm": (_I, [_P, _P, _P, _P, ctypes.c_float, _P, _P, _I, _I, ctypes.c_uint, _P]),
    "q8_choose": (_I, [_P, _I, _P, _P, _I, _P, _I, _I, _P]),
}


class _Part(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("y", ctypes.c_void_p), ("N", ctypes.c_int)]

_lib = None


class Q8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = lib().q8_status_string(status).decode()
        if status == 5:
            detail += f" (cudaError {lib().q8_last_cuda_error()})"
        super().__init__(f"{where}: {_STATUS.get(status, status)}: {detail}")


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded library; raises when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libq8gemv is not built ({_LIB_PATH} missing); run "
                               "`python -m q8_block_quantized_gemv_gb300.build`")
        handle = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise Q8Error(status, where)


_INT_MAX = 2 ** 31 - 1  # the library's sizes and row pitches are 32-bit: ctypes would pass the low bits of a larger one


def padded_n(N: int) -> int:
    return lib().q8_padded_n(N)


def status_string(status: int) -> str:
    return lib().q8_status_string(status).decode()


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_raw_stream = None


def _stream_of(stream, device):
    """The handle of ``stream``, or of the device's current stream: torch's own look-up where it has it, a tenth of the
    time that making a Stream object for it takes."""
    global _raw_stream
    if stream is not None:
        return _stream_handle(stream)
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(device.index)


def _new(shape, dtype, device, stream=None, zeroed=False, returned=True):
    """A tensor for a call that runs on ``stream`` (None: the current stream).  It is allocated, and zeroed, on that
    stream: memory that other work of the current stream may still be using does not go to a kernel that nothing orders
    behind it.  A returned tensor may be used on the current stream as well, once that waits for ``stream``, and freed."""
    import torch
    make = torch.zeros if zeroed else torch.empty
    if stream is None or _stream_handle(stream) == _stream_of(None, device):
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(_stream_handle(stream), device=device)):
        out = make(shape, dtype=dtype, device=device)
    if returned:
        out.record_stream(torch.cuda.current_stream(device))
    return out


def tiled_n(N: int) -> int:
    return lib().q8_tiled_n(N)


class QuantAct:
    """The quantized form of an activation (q8_quantize_act): one uint8 CUDA buffer of ``act_bytes(m, K)`` bytes
    holding int8 values [m, K] followed by fp32 scales [m, K/32].  Pass it as ``x`` to any product function (tiled
    weights only)."""

    def __init__(self, buf, m: int, K: int):
        self.buf, self.shape = buf, (m, K)

    @property
    def device(self):
        return self.buf.device

    @property
    def is_cuda(self):
        return self.buf.is_cuda

    def data_ptr(self) -> int:
        return self.buf.data_ptr()

    def values(self):
        """int8 [m, K] view of the codes."""
        import torch
        m, K = self.shape
        return self.buf[: m * K].view(torch.int8).view(m, K)

    def scales(self):
        """fp32 [m, K/32] view of the scales."""
        import torch
        m, K = self.shape
        return self.buf[m * K:].view(torch.float32).view(m, K // Q8_BLOCK)


def act_bytes(m: int, K: int) -> int:
    return int(lib().q8_act_bytes(m, K))


def quantize_act(x, out: QuantAct | None = None, stream=None) -> QuantAct:
    """bf16 x [m, K] (CUDA, contiguous) -> its quantized form (q8_quantize_act)."""
    import torch
    if not x.is_cuda or x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D bfloat16 CUDA tensor")
    m, K = x.shape
    nbytes = act_bytes(m, K)
    if nbytes < 0:
        raise ValueError("K must be a positive multiple of 32")
    if out is None:
        out = QuantAct(_new((nbytes,), torch.uint8, x.device, stream), m, K)
    elif out.shape != (m, K) or out.buf.numel() != nbytes:
        raise ValueError("out must be a QuantAct of the same shape")
    _check(lib().q8_quantize_act(x.data_ptr(), out.data_ptr(), m, K, _stream_handle(stream)), "q8_quantize_act")
    return out


def _check_operands(x, q, s, N, tiled=False):
    import torch
    if isinstance(x, QuantAct):
        if not tiled:
            raise ValueError("a quantized activation takes tiled weights")
        if not (q.is_cuda and s.is_cuda and x.is_cuda):
            raise ValueError("x, q and s must be CUDA tensors")
        if q.dtype != torch.int8 or s.dtype != torch.float32 or not (q.is_contiguous() and s.is_contiguous()):
            raise TypeError("q must be contiguous int8 and s contiguous float32")
        m, K = x.shape
    else:
        if not (x.is_cuda and q.is_cuda and s.is_cuda):
            raise ValueError("x, q and s must be CUDA tensors")
        if x.dtype != torch.bfloat16 or q.dtype != torch.int8 or s.dtype != torch.float32:
            raise TypeError("x must be bfloat16, q int8 and s float32")
        if not (x.is_contiguous() and q.is_contiguous() and s.is_contiguous()):
            raise ValueError("x, q and s must be contiguous")
        if x.dim() != 2:
            raise ValueError("x must be 2-D [m, K]")
        m, K = x.shape
    Np = padded_n(N) if N > 0 else -1
    if tiled:
        Nt = tiled_n(N) if N > 0 else -1
        if q.numel() != K * Nt or s.numel() != (K // Q8_BLOCK) * Nt:
            raise ValueError(f"tiled q must hold K * Nt = {K * Nt} values and s (K/32) * Nt scales")
    elif q.shape != (K, Np) or s.shape != (K // Q8_BLOCK, Np):
        raise ValueError(f"q must be [K, Np] = [{K}, {Np}] and s [K/32, Np]; got {tuple(q.shape)}, {tuple(s.shape)}")
    return m, K, Np


FLAG_CONSTANT_WEIGHTS = 1
FLAG_TILED = 2
FLAG_Q8_ACT = 4


def _flags(constant_weights, tiled, x=None):
    return ((FLAG_CONSTANT_WEIGHTS if constant_weights else 0) | (FLAG_TILED if tiled else 0)
            | (FLAG_Q8_ACT if isinstance(x, QuantAct) else 0))


def gemv(x, q, s, N: int, y=None, variant: str = "auto", constant_weights: bool = False, tiled: bool = False,
         stream=None):
    """y = x . W over the Q8_0 weight (q, s); returns y, fp32 [m, Np] (columns N .. Np-1 are 0).

    constant_weights: nothing enqueued earlier on the stream, other than :func:`tile_device`, writes q or s
    (Q8_FLAG_CONSTANT_WEIGHTS), so the kernel may stream them before the previous kernel finishes.  tiled: q and s are in the tiled layout
    (:func:`tile_device`, Q8_FLAG_TILED)."""
    import torch
    m, K, Np = _check_operands(x, q, s, N, tiled)
    if y is None:
        y = _new((m, Np), torch.float32, x.device, stream)
    elif y.dtype != torch.float32 or y.shape != (m, Np) or not y.is_contiguous() or not y.is_cuda:
        raise ValueError("y must be a contiguous fp32 CUDA tensor [m, Np]")
    _check(lib().q8_gemv_ex(x.data_ptr(), q.data_ptr(), s.data_ptr(), y.data_ptr(), m, K, N, VARIANTS[variant],
                            _flags(constant_weights, tiled, x), _stream_handle(stream)), "q8_gemv")
    return y


def gemv_argmax(x, q, s, N: int, idx=None, logits=None, constant_weights: bool = False, tiled: bool = False,
                stream=None):
    """The product and its first-maximum arg-max per row: returns idx, int64 [m] (0-based).

    ``logits``: None (not stored) or a contiguous fp32 [m, Np] CUDA tensor that receives y.
    """
    import torch
    m, K, Np = _check_operands(x, q, s, N, tiled)
    if idx is None:
        idx = _new((m,), torch.int64, x.device, stream)
    elif idx.dtype != torch.int64 or idx.numel() < m or not idx.is_contiguous() or not idx.is_cuda:
        raise ValueError("idx must be a contiguous int64 CUDA tensor of m elements")
    lp = None
    if logits is not None:
        if logits.dtype != torch.float32 or logits.shape != (m, Np) or not logits.is_contiguous():
            raise ValueError("logits must be a contiguous fp32 CUDA tensor [m, Np]")
        lp = logits.data_ptr()
    _check(lib().q8_gemv_argmax_ex(x.data_ptr(), q.data_ptr(), s.data_ptr(), idx.data_ptr(), lp, m, K, N,
                                   _flags(constant_weights, tiled, x), _stream_handle(stream)), "q8_gemv_argmax")
    return idx


def tile(q, s, N: int):
    """Host: row-major (q [K, Np], s [K/32, Np]) numpy arrays -> the tiled layout (qt int8 [K * Nt], st fp32
    [K/32 * Nt]) (q8_tile)."""
    q = np.ascontiguousarray(q, dtype=np.int8)
    s = np.ascontiguousarray(s, dtype=np.float32)
    K = q.shape[0]
    Nt = tiled_n(N) if N > 0 else 1
    qt = np.empty(max(K * Nt, 1), dtype=np.int8)
    st = np.empty(max((K // Q8_BLOCK) * Nt, 1), dtype=np.float32)
    _check(lib().q8_tile(q.ctypes.data, s.ctypes.data, K, N, qt.ctypes.data, st.ctypes.data), "q8_tile")
    return qt, st


def tile_device(q, s, N: int, stream=None):
    """Device: row-major CUDA tensors (q [K, Np] int8, s [K/32, Np] fp32) -> tiled CUDA tensors (q8_tile_device)."""
    import torch
    K = q.shape[0]
    Nt = tiled_n(N)
    qt = _new((K * Nt,), torch.int8, q.device, stream)
    st = _new(((K // Q8_BLOCK) * Nt,), torch.float32, q.device, stream)
    _check(lib().q8_tile_device(q.data_ptr(), s.data_ptr(), K, N, qt.data_ptr(), st.data_ptr(),
                                _stream_handle(stream)), "q8_tile_device")
    return qt, st


def gemv_parts(x, weights, ys=None, constant_weights: bool = False, tiled: bool = False, stream=None):
    """Several products of one activation in one call (q8_gemv_parts): weights is a list of (q, s, N); returns the
    list of outputs y_p, fp32 [m, Np_p]."""
    import torch
    if not weights or len(weights) > 8:
        raise ValueError("1 to 8 parts")
    m, K = x.shape
    arr = (_Part * len(weights))()
    outs = []
    for i, (q, s, N) in enumerate(weights):
        _check_operands(x, q, s, N, tiled)
        Np = padded_n(N)
        y = ys[i] if ys is not None else _new((m, Np), torch.float32, x.device, stream)
        if y.dtype != torch.float32 or y.shape != (m, Np) or not y.is_contiguous() or not y.is_cuda:
            raise ValueError("each y must be a contiguous fp32 CUDA tensor [m, Np]")
        arr[i] = _Part(q.data_ptr(), s.data_ptr(), y.data_ptr(), N)
        outs.append(y)
    _check(lib().q8_gemv_parts(x.data_ptr(), ctypes.cast(arr, ctypes.c_void_p), len(weights), m, K,
                               _flags(constant_weights, tiled, x), _stream_handle(stream)), "q8_gemv_parts")
    return outs


def plan_launches(m: int, K: int, Ns, tiled: bool = True, q8_act: bool = False) -> int:
    """How many product kernels a gemv / gemv_argmax / gemv_parts call of these sizes launches on the current device
    (q8_plan_launches): 1, or 2 when the planner splits it in two."""
    arr = (ctypes.c_int * len(Ns))(*[int(n) for n in Ns])
    flags = (FLAG_TILED if tiled else 0) | (FLAG_Q8_ACT if q8_act else 0)
    n = int(lib().q8_plan_launches(int(m), int(K), ctypes.cast(arr, ctypes.c_void_p), len(Ns), flags))
    if n < 0:
        raise Q8Error(-n, "q8_plan_launches")
    return n


def plan_glu_launches(m: int, K: int, N: int, q8_act: bool = False) -> int:
    """How many kernels a gemv_glu call of these sizes launches on the current device (q8_plan_glu_launches)."""
    n = int(lib().q8_plan_glu_launches(int(m), int(K), int(N), FLAG_TILED | (FLAG_Q8_ACT if q8_act else 0)))
    if n < 0:
        raise Q8Error(-n, "q8_plan_glu_launches")
    return n


def _q8_out(out_q8, m, Np, device, stream):
    import torch
    if out_q8 is None:
        return QuantAct(_new((act_bytes(m, Np),), torch.uint8, device, stream), m, Np)
    if out_q8.shape != (m, Np) or out_q8.buf.numel() != act_bytes(m, Np):
        raise ValueError("out_q8 must be a QuantAct of [m, Np]")
    return out_q8


def gemv_glu(x, gate, up, N: int, out=None, out_bf16=None, want=("f32",), constant_weights: bool = False,
             stream=None, out_q8=None):
    """The gated pair (q8_gemv_glu_ex, SwiGLU): silu(x.Wg) * (x.Wu) with both weights tiled; gate and up are (q, s).

    ``want``: which outputs to allocate when not given -- "f32" (fp32 [m, Np]), "bf16" (bf16 [m, Np]) and/or "q8"
    (the quantized form of the bf16 output, a QuantAct of [m, Np]).  Returns (out, out_bf16), either None when not
    requested, or (out, out_bf16, out_q8) when "q8" is wanted or out_q8 given."""
    import torch
    m, K, Np = _check_operands(x, gate[0], gate[1], N, True)
    _check_operands(x, up[0], up[1], N, True)
    if out is None and "f32" in want:
        out = _new((m, Np), torch.float32, x.device, stream)
    if out_bf16 is None and "bf16" in want:
        out_bf16 = _new((m, Np), torch.bfloat16, x.device, stream)
    q8out = out_q8 is not None or "q8" in want
    if q8out:
        out_q8 = _q8_out(out_q8, m, Np, x.device, stream)
    if out is not None and (out.dtype != torch.float32 or out.shape != (m, Np) or not out.is_contiguous()):
        raise ValueError("out must be a contiguous fp32 CUDA tensor [m, Np]")
    if out_bf16 is not None and (out_bf16.dtype != torch.bfloat16 or out_bf16.shape != (m, Np)
                                 or not out_bf16.is_contiguous()):
        raise ValueError("out_bf16 must be a contiguous bf16 CUDA tensor [m, Np]")
    _check(lib().q8_gemv_glu_ex(x.data_ptr(), gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(),
                                up[1].data_ptr(), out.data_ptr() if out is not None else None,
                                out_bf16.data_ptr() if out_bf16 is not None else None,
                                out_q8.data_ptr() if q8out else None, m, K, N,
                                _flags(constant_weights, True, x), _stream_handle(stream)), "q8_gemv_glu")
    return (out, out_bf16, out_q8) if q8out else (out, out_bf16)


def gemv_residual_norm(x, q, s, N: int, residual, gamma, eps: float, h=None, out_bf16=None,
                       constant_weights: bool = False, stream=None, want=("bf16",), out_q8=None):
    """A projection followed by the residual add and the following RMS norm (q8_gemv_residual_norm_ex), tiled weight:
    h = residual + x.W, out = h / sqrt(mean(h^2) + eps) * gamma.  Returns (h fp32 [m, Np], out bf16 [m, Np]), or
    (h, out_bf16 or None, out_q8) when ``want`` holds "q8" or out_q8 is given (the quantized form of the bf16 rows);
    ``h`` may be ``residual`` (in place)."""
    import torch
    m, K, Np = _check_operands(x, q, s, N, True)
    if residual.dtype != torch.float32 or residual.shape != (m, Np) or not residual.is_contiguous():
        raise ValueError("residual must be a contiguous fp32 CUDA tensor [m, Np]")
    if gamma.dtype != torch.float32 or gamma.numel() < N or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous fp32 CUDA tensor of at least N values")
    if h is None:
        h = _new((m, Np), torch.float32, x.device, stream)
    if out_bf16 is None and "bf16" in want:
        out_bf16 = _new((m, Np), torch.bfloat16, x.device, stream)
    q8out = out_q8 is not None or "q8" in want
    if q8out:
        out_q8 = _q8_out(out_q8, m, Np, x.device, stream)
    _check(lib().q8_gemv_residual_norm_ex(x.data_ptr(), q.data_ptr(), s.data_ptr(), residual.data_ptr(),
                                          gamma.data_ptr(), float(eps), h.data_ptr(),
                                          out_bf16.data_ptr() if out_bf16 is not None else None,
                                          out_q8.data_ptr() if q8out else None, m, K, N,
                                          _flags(constant_weights, True, x), _stream_handle(stream)),
           "q8_gemv_residual_norm")
    return (h, out_bf16, out_q8) if q8out else (h, out_bf16)


# Planner overrides (q8_set_tuning): the K split (0 = the planner's, 1..8 forced), the prefill GEMM (-1 = the
# planner's, 0 = row groups, 1 = GEMM), the residual norm's route (0 = own launch, 1 = the one-launch fold) and the
# two-launch split of plain products (1 = where the planner finds one, 0 = never).
TUNING = {"ksplit": 0, "gemm": 1, "norm_fold": 2, "split": 3}


def set_tuning(option: str, value: int) -> None:
    """Set a process-wide planner override (q8_set_tuning) for tests and benchmarks."""
    _check(lib().q8_set_tuning(TUNING[option], int(value)), "q8_set_tuning")


def get_tuning(option: str) -> int:
    """The current value of a planner override (q8_get_tuning)."""
    return int(lib().q8_get_tuning(TUNING[option]))


class tuning:
    """Context manager: ``with tuning(ksplit=4): ...`` sets overrides and restores the previous values on exit."""

    def __init__(self, **overrides):
        self.overrides, self.saved = overrides, {}

    def __enter__(self):
        for k, v in self.overrides.items():
            self.saved.setdefault(k, get_tuning(k))
            set_tuning(k, v)
        return self

    def __exit__(self, *exc):
        for k, v in self.saved.items():
            set_tuning(k, v)


def gemv_residual_norm_noalloc(x, q, s, N: int, residual, gamma, eps: float, h, out_bf16,
                               constant_weights: bool = False, stream=None):
    """q8_gemv_residual_norm_noalloc: the residual add and RMS norm as one launch whose scratch is the library's own
    static counters (no device allocation by anyone).  h and out_bf16 must be given (h may be ``residual``); calls
    that overlap on the GPU race on the shared counters.  Returns (h, out_bf16)."""
    import torch
    m, K, Np = _check_operands(x, q, s, N, True)
    if residual.dtype != torch.float32 or residual.shape != (m, Np) or not residual.is_contiguous():
        raise ValueError("residual must be a contiguous fp32 CUDA tensor [m, Np]")
    if gamma.dtype != torch.float32 or gamma.numel() < N or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous fp32 CUDA tensor of at least N values")
    if h.dtype != torch.float32 or h.shape != (m, Np) or not h.is_contiguous():
        raise ValueError("h must be a contiguous fp32 CUDA tensor [m, Np]")
    if out_bf16.dtype != torch.bfloat16 or out_bf16.shape != (m, Np) or not out_bf16.is_contiguous():
        raise ValueError("out_bf16 must be a contiguous bf16 CUDA tensor [m, Np]")
    _check(lib().q8_gemv_residual_norm_noalloc(x.data_ptr(), q.data_ptr(), s.data_ptr(), residual.data_ptr(),
                                               gamma.data_ptr(), float(eps), h.data_ptr(), out_bf16.data_ptr(), m, K,
                                               N, _flags(constant_weights, True, x), _stream_handle(stream)),
           "q8_gemv_residual_norm_noalloc")
    return h, out_bf16


class _KV(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("page_stride", ctypes.c_int64),
                ("pages", _I), ("heads", _I), ("page_size", _I), ("dim", _I)]


FLAG_ROPE_INTERLEAVED = 1


class KVCache:
    """A paged key-value cache (q8_kv_cache): k and v, CUDA tensors [pages, heads, page_size, dim], bfloat16, or int8
    with k_scale and v_scale, float32 [pages, heads, page_size, dim / 32].  Pages may be apart (views of a larger
    allocation), everything inside a page is contiguous.  :meth:`empty` allocates one."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        q8 = k_scale is not None
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must be [pages, heads, page_size, dim]")
        pages, heads, page_size, dim = k.shape
        dense = heads * page_size * dim
        stride = k.stride(0) if pages > 1 else dense
        for x, shape, ps in ((k, k.shape, stride), (v, k.shape, stride)) + (
                ((k_scale, (*k.shape[:3], dim // Q8_BLOCK), stride // Q8_BLOCK),
                 (v_scale, (*k.shape[:3], dim // Q8_BLOCK), stride // Q8_BLOCK)) if q8 or v_scale is not None else ()):
            if x is None or not x.is_cuda or x.get_device() != k.get_device() or tuple(x.shape) != tuple(shape):
                raise ValueError("k, v and the scales must be CUDA tensors of one device, the scales [..., dim / 32]")
            if pages and not x[0].is_contiguous() or (pages > 1 and x.stride(0) != ps):
                raise ValueError("a page must be contiguous, and the pages of k, v and the scales equally far apart")
        want = torch.int8 if q8 else torch.bfloat16
        if k.dtype != want or v.dtype != want or (q8 and (k_scale.dtype, v_scale.dtype) != (torch.float32,) * 2):
            raise TypeError("k and v must be bfloat16, or int8 with float32 scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.dim, self.device = pages, heads, page_size, dim, k.device
        self._c = _KV(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if q8 else None,
                      v_scale.data_ptr() if q8 else None, stride, pages, heads, page_size, dim)
        self._ref, self._index = ctypes.addressof(self._c), k.get_device()

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, dim: int, dtype: str = "bf16", device="cuda"):
        """A zeroed cache of the given type, "bf16" or "q8"."""
        import torch
        shape = (pages, heads, page_size, dim)
        if dtype == "bf16":
            return cls(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        if dtype != "q8":
            raise ValueError("dtype must be \"bf16\" or \"q8\"")
        sshape = (pages, heads, page_size, dim // Q8_BLOCK)
        return cls(*(torch.zeros(shape, dtype=torch.int8, device=device) for _ in range(2)),
                   *(torch.zeros(sshape, dtype=torch.float32, device=device) for _ in range(2)))


# The tensors of one call are on one device: `index` is the cache's, or the first tensor's (-1: on the CPU).

def _ints(name, t, index, n=None):
    import torch
    if index < 0 or t.get_device() != index or t.dtype != torch.int32 or not t.is_contiguous() or \
            (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor" + (f" of {n} values" if n is not None else "") +
                         ", on the device of the others")
    return t.data_ptr()


def _table_of(table, R, index):
    import torch
    shape = table.shape
    if table.get_device() != index or table.dtype != torch.int32 or len(shape) != 2 or shape[0] != R or \
            (shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"the block table must be an int32 CUDA tensor [{R}, width] with unit column stride, on the device "
                         "of the others")
    pitch = table.stride(0) if R > 1 else shape[1]
    if pitch > _INT_MAX or R > _INT_MAX:
        raise ValueError("the block table's rows are more than 2^31 - 1, or as far apart")
    return table.data_ptr(), shape[1], pitch


def kv_slots(cached, fresh, table, free_pages, page_size: int, rows: int, head=None, stream=None, out=None):
    """Block tables and slot maps of one step (q8_kv_slots): request r has cached[r] tokens in the cache and fresh[r]
    new ones (int32 [R]); new pages come from free_pages[head:] and are written into ``table`` (int32 [R, width]) in
    place.  Returns a dict of CUDA tensors: table, lens int32 [R], row_start int32 [R + 1], positions int32 [rows],
    slots int64 [rows] (rows past the total: -1), head int32 [1], the next step's.  ``out``: such a dict to write."""
    import torch
    R, index, dev = cached.numel(), cached.get_device(), cached.device
    c, f = _ints("cached", cached, index), _ints("fresh", fresh, index, R)
    t, width, pitch = _table_of(table, R, index)
    if out is None:
        i32 = torch.int32  # tensors of their own: cheaper than views of one
        lens, starts = _new(R, i32, dev, stream), _new(R + 1, i32, dev, stream)
        positions, next_head = _new(rows, i32, dev, stream), _new(1, i32, dev, stream)
        slots = _new(rows, torch.int64, dev, stream)
        out = {"table": table, "lens": lens, "row_start": starts, "positions": positions, "slots": slots,
               "head": next_head}
        lp, sp, pp, hp = lens.data_ptr(), starts.data_ptr(), positions.data_ptr(), next_head.data_ptr()
    else:
        slots = out["slots"]
        if slots.dtype != torch.int64 or slots.numel() != rows or not slots.is_contiguous() \
                or slots.get_device() != index or out["table"] is not table:
            raise ValueError("out must hold this table and contiguous CUDA tensors of the sizes kv_slots returns")
        lp, sp = _ints("lens", out["lens"], index, R), _ints("row_start", out["row_start"], index, R + 1)
        hp, pp = _ints("head", out["head"], index, 1), _ints("positions", out["positions"], index, rows)
    st = lib().q8_kv_slots(c, f, R, page_size, _ints("free_pages", free_pages, index), free_pages.numel(),
                           None if head is None else _ints("head", head, index, 1), t, width, pitch, rows, lp, sp, pp,
                           slots.data_ptr(), hp, _stream_of(stream, dev))
    if st:
        raise Q8Error(st, "q8_kv_slots")
    return out


def rope_table(positions: int, rotary_dim: int, base: float = 10000.0, scaling=None, device="cuda"):
    """The rotation table of q8_rope_append: fp32 [positions, rotary_dim], row p holding cos(p f_i) for the
    rotary_dim / 2 pairs i, then sin(p f_i), with f_i = base ** (-2 i / rotary_dim); computed in fp64 on the host, so
    the angles of long positions keep their precision.  ``scaling`` stretches it for contexts longer than trained:

    * ("linear", s): positions divided by s (position interpolation);
    * ("ntk", s): base times s ** (rotary_dim / (rotary_dim - 2)): the slowest pair is stretched by s, the fastest kept;
    * ("parts", s, trained[, fast, slow[, amplitude]]): pair by pair, by the turns trained * f_i / (2 pi) it makes over
      the trained length: more than ``fast`` (32) turns keep f_i, fewer than ``slow`` (1) take f_i / s, a linear ramp
      over the pair index between; cos and sin times ``amplitude`` (0.1 ln s + 1)."""
    import torch
    if rotary_dim % 2 or rotary_dim < 2 or positions < 1:
        raise ValueError("rotary_dim must be even and positive, positions at least 1")
    numbers = [float(x) for x in (base, *(scaling[1:] if scaling else ()))]
    if not all(np.isfinite(x) and x > 0 for x in numbers):
        raise ValueError("base and the numbers of scaling must be finite and positive")
    if scaling and not {"linear": 2, "ntk": 2, "parts": 3}.get(scaling[0], 0) <= len(scaling):
        raise ValueError(f"scaling {scaling[0]!r} needs more numbers")
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    amplitude = 1.0
    kind = scaling[0] if scaling else None
    if kind == "ntk":
        base = base * float(scaling[1]) ** (rotary_dim / (rotary_dim - 2)) if rotary_dim > 2 else base
    f = base ** (-2.0 * i / rotary_dim)
    if kind == "linear":
        f = f / float(scaling[1])
    elif kind == "parts":
        s, trained = float(scaling[1]), float(scaling[2])
        fast, slow = (float(scaling[3]), float(scaling[4])) if len(scaling) > 4 else (32.0, 1.0)
        amplitude = float(scaling[5]) if len(scaling) > 5 else 0.1 * np.log(s) + 1.0 if s > 1 else 1.0
        at = [rotary_dim * np.log(trained / (2 * np.pi * turns)) / (2 * np.log(base)) for turns in (fast, slow)]
        low, high = max(np.floor(at[0]), 0.0), min(np.ceil(at[1]), rotary_dim - 1.0)
        ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        f = f * (1.0 - ramp) + f / s * ramp
    elif kind not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling[0]!r}")
    angle = np.arange(positions, dtype=np.float64)[:, None] * f
    both = np.concatenate([np.cos(angle), np.sin(angle)], axis=1) * amplitude
    return torch.from_numpy(both.astype(np.float32)).to(device)


def _rows2(name, x, dtype, cols, index):
    shape = x.shape
    if x.get_device() != index or x.dtype != dtype or len(shape) != 2 or shape[1] < cols or x.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D {dtype} CUDA tensor of at least {cols} columns, unit column stride, on the "
                         "cache's device")
    pitch = x.stride(0) if shape[0] > 1 else cols  # one row has no pitch
    if pitch > _INT_MAX or shape[0] > _INT_MAX:
        raise ValueError(f"the rows of {name} are more than 2^31 - 1, or as far apart")
    return x.data_ptr(), pitch


def rope_append(q, k, v, cache: KVCache, positions, slots, table=None, q_heads: int | None = None,
                interleaved: bool = False, q_gamma=None, k_gamma=None, eps: float = 1e-6, out=None, stream=None):
    """Norms of q and k per head, their rotation, and the append of k and v to the cache (q8_rope_append).  q, k, v:
    the products' fp32 outputs [rows, >= heads * dim] (q_heads defaults to q's columns / dim); positions int32 [rows],
    slots int64 [rows] (:func:`kv_slots`); ``table``: :func:`rope_table`, its width the rotated part of a head (None:
    no rotation).  Returns q, bf16 [rows, q_heads * dim]."""
    import torch
    dim, f32, index = cache.dim, torch.float32, cache._index
    if q_heads is None:
        q_heads = q.shape[-1] // dim
    rows, n, m = q.shape[0], q_heads * dim, cache.heads * dim
    qp, ldq = _rows2("q", q, f32, max(n, 1), index)
    kp, ldk = _rows2("k", k, f32, m, index)
    vp, ldv = _rows2("v", v, f32, m, index)
    if k.shape[0] != rows or v.shape[0] != rows:
        raise ValueError("q, k and v must have the same rows")
    if slots.get_device() != index or slots.dtype != torch.int64 or slots.numel() != rows or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int64 CUDA tensor of one value a row")
    pos = _ints("positions", positions, index, rows)
    for g in (q_gamma, k_gamma):
        if g is not None and (g.get_device() != index or g.dtype != f32 or g.numel() != dim or not g.is_contiguous()):
            raise ValueError("a gamma must be a contiguous fp32 CUDA tensor of dim values")
    tp, limit, rot = None, 0, 0
    if table is not None:
        if table.get_device() != index or table.dtype != f32 or table.dim() != 2 or not table.is_contiguous():
            raise ValueError("table must be a contiguous fp32 CUDA tensor [positions, rotary_dim]")
        tp, (limit, rot) = table.data_ptr(), table.shape
    if out is None:
        out = _new((rows, n), torch.bfloat16, q.device, stream)
        op, ldo = out.data_ptr(), n
    else:
        if out.shape[0] != rows:
            raise ValueError("out must have q's rows")
        op, ldo = _rows2("out", out, torch.bfloat16, max(n, 1), index)
    if rows == 0:
        return out
    st = lib().q8_rope_append(qp, ldq, kp, ldk, vp, ldv, None if q_gamma is None else q_gamma.data_ptr(),
                              None if k_gamma is None else k_gamma.data_ptr(), eps, tp, limit, rot, pos,
                              slots.data_ptr(), op, ldo, cache._ref, rows, q_heads,
                              FLAG_ROPE_INTERLEAVED if interleaved else 0, _stream_of(stream, cache.device))
    if st:
        raise Q8Error(st, "q8_rope_append")
    return out


_workspace_bytes = 0


def attn_workspace(device="cuda"):
    """A zeroed workspace for attn_decode and attn_prefill (q8_attn_workspace_bytes); keep one per stream."""
    import torch
    global _workspace_bytes
    _workspace_bytes = int(lib().q8_attn_workspace_bytes())
    return torch.zeros((_workspace_bytes,), dtype=torch.uint8, device=device)


def _attn(q, cache, R, table, lens, q_heads, scale, out, workspace, stream):
    import torch
    shape, index = q.shape, cache._index
    if q_heads is None:
        q_heads = shape[-1] // cache.dim
    n = q_heads * cache.dim
    qp, ldq = _rows2("q", q, torch.bfloat16, max(n, 1), index)
    tp, width, pitch = _table_of(table, R, index)
    if out is None:
        out = _new((shape[0], n), torch.bfloat16, q.device, stream)
        op, ldo = out.data_ptr(), n
    else:
        if out.shape[0] != shape[0]:
            raise ValueError("out must have q's rows")
        op, ldo = _rows2("out", out, torch.bfloat16, max(n, 1), index)
    if workspace is None:
        workspace = _new((int(lib().q8_attn_workspace_bytes()),), torch.uint8, q.device, stream, zeroed=True,
                         returned=False)  # of this call alone: its stream's again when the call returns
    elif workspace.get_device() != index or not workspace.is_contiguous() or \
            workspace.nbytes < (_workspace_bytes or lib().q8_attn_workspace_bytes()):
        raise ValueError("workspace must come from attn_workspace")
    return (qp, ldq, cache._ref, tp, width, pitch, _ints("lens", lens, index, R), op, ldo, q_heads,
            cache.dim ** -0.5 if scale is None else scale, out, workspace)


def _int32(n):
    """A window's or sinks' length as the library's 32-bit int: past 2^31 they reach any position all the same."""
    return max(-1, min(n, 0x7FFFFFFF))


def attn_decode(q, cache: KVCache, table, lens, q_heads: int | None = None, scale: float | None = None,
                window: int = 0, sinks: int = 0, out=None, workspace=None, stream=None):
    """Attention of one new token a request over its pages (q8_attn_decode): q bf16 [R, >= q_heads * dim], block table
    int32 [R, width], lens int32 [R] (the new token included; 0: an idle row, which gets zeros).  ``window``: keys that
    far back or more are hidden (0: none), but for the first ``sinks``.  ``scale`` defaults to dim ** -0.5.
    ``workspace``: :func:`attn_workspace`, one per stream (None: allocated and zeroed for this call, on its stream).  Returns bf16
    [R, q_heads * dim], the output projection's activation."""
    R = q.shape[0]
    qp, ldq, kv, tp, width, pitch, lp, op, ldo, q_heads, scale, out, workspace = \
        _attn(q, cache, R, table, lens, q_heads, scale, out, workspace, stream)
    if R == 0:
        return out
    st = lib().q8_attn_decode(qp, ldq, kv, tp, width, pitch, lp, op, ldo, R, q_heads, scale, _int32(window),
                              _int32(sinks), workspace.data_ptr(), _stream_of(stream, cache.device))
    if st:
        raise Q8Error(st, "q8_attn_decode")
    return out


def attn_prefill(q, cache: KVCache, table, lens, row_start, q_heads: int | None = None, scale: float | None = None,
                 window: int = 0, sinks: int = 0, out=None, workspace=None, stream=None):
    """Causal attention of a chunk of new tokens over the pages (q8_attn_prefill): rows row_start[r] .. row_start[r+1]
    of q are the last tokens of request r, whose keys are in the cache already; row_start int32 [R + 1], lens int32
    [R].  Rows past row_start[R] get zeros.  Other arguments as :func:`attn_decode`."""
    R, rows = lens.numel(), q.shape[0]
    qp, ldq, kv, tp, width, pitch, lp, op, ldo, q_heads, scale, out, workspace = \
        _attn(q, cache, R, table, lens, q_heads, scale, out, workspace, stream)
    if rows == 0:
        return out
    st = lib().q8_attn_prefill(qp, ldq, kv, tp, width, pitch, lp, _ints("row_start", row_start, cache._index, R + 1), op, ldo, rows,
                               R, q_heads, scale, _int32(window), _int32(sinks), workspace.data_ptr(),
                               _stream_of(stream, cache.device))
    if st:
        raise Q8Error(st, "q8_attn_prefill")
    return out


class _W4(ctypes.Structure):
    _fields_ = [("w", _P), ("N", _I), ("group", _I), ("flags", ctypes.c_uint)]


class Weight4:
    """A weight of 4-bit codes with group scales, laid out for the products (q8_w4_tile_device): value = scale * (code -
    zero).  From CUDA tensors as a checkpoint has them: ``codes`` uint8 [K/2, N] (row 2i in the low half of byte row i),
    ``scales`` float16 or bfloat16 [K/group, N] with group 32, 64 or 128, ``zeros`` uint8 [K/group, N] of 0..127 (None: 8
    everywhere).  Keeps its own copy, ``buf``; :func:`tile4` lays it out on the host, :meth:`of_tiled` takes that.  Products on the
    same stream may take it with ``constant_weights`` at once; other work that writes ``buf`` (a copy into a tensor given to
    :meth:`of_tiled`) has to have ended before such a call is made."""

    def __init__(self, codes, scales, zeros=None, stream=None):
        import torch
        for name, t in (("codes", codes), ("scales", scales), ("zeros", zeros)):
            if t is not None and (not t.is_cuda or t.get_device() != codes.get_device() or t.dim() != 2
                                  or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous 2-D CUDA tensor, on the device of the others")
        if codes.dtype != torch.uint8 or scales.dtype not in (torch.float16, torch.bfloat16) or \
                (zeros is not None and zeros.dtype != torch.uint8):
            raise TypeError("codes and zeros must be uint8, scales float16 or bfloat16")
        K, N = 2 * codes.shape[0], codes.shape[1]
        groups = scales.shape[0]
        if scales.shape[1] != N or (zeros is not None and zeros.shape != scales.shape) or not groups or K % groups:
            raise ValueError("scales and zeros must be [K / group, N], codes [K / 2, N]")
        flags = (FLAG_W4_ZEROS if zeros is not None else 0) | (FLAG_W4_BF16 if scales.dtype == torch.bfloat16 else 0)
        size = _w4_bytes(K, N, K // groups, flags)
        if size < 0:
            raise ValueError("a group is 32, 64 or 128 rows; K is at most 2^31 - 128, and N, rounded up to 32, less than 2^31")
        self._keep(_new((size,), torch.uint8, codes.device, stream), K, N, K // groups, flags)
        _check(lib().q8_w4_tile_device(codes.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(), K,
                                       N, self.group, flags, self.buf.data_ptr(), _stream_of(stream, codes.device)),
               "q8_w4_tile_device")

    @classmethod
    def of_tiled(cls, buf, K: int, N: int, group: int, zeros: bool = False, bf16_scales: bool = False):
        """A weight whose tiled form (uint8 CUDA tensor, 16-byte aligned) is at hand."""
        import torch
        flags = (FLAG_W4_ZEROS if zeros else 0) | (FLAG_W4_BF16 if bf16_scales else 0)
        size = _w4_bytes(K, N, group, flags)
        if size < 0 or not buf.is_cuda or buf.dtype != torch.uint8 or not buf.is_contiguous() or buf.numel() != size:
            raise ValueError(f"buf must be a contiguous uint8 CUDA tensor of {size} bytes")
        self = cls.__new__(cls)
        self._keep(buf, K, N, group, flags)
        return self

    def _keep(self, buf, K, N, group, flags):
        self.buf, self.K, self.N, self.Np, self.group, self.flags = buf, K, N, padded_n(N), group, flags
        self.device, self._index = buf.device, buf.get_device()
        self._c = _W4(buf.data_ptr(), N, group, flags)
        self._ref, self._packed = ctypes.addressof(self._c), bytes(self._c)
        # what every call needs, at hand: looking it up took a fifth of a small call's time
        import torch
        self._bf16, self._f32, self._empty = torch.bfloat16, torch.float32, torch.empty


FLAG_W4_ZEROS = 1
FLAG_W4_BF16 = 2


def _w4_bytes(K, N, group, flags):
    """q8_w4_bytes; -1 for sizes that are not the library's, those beyond its 32 bits among them."""
    return int(lib().q8_w4_bytes(K, N, group, flags)) if all(0 < n <= _INT_MAX for n in (K, N, group)) else -1


def tile4(codes, scales, zeros=None, bf16_scales: bool = False):
    """Host: numpy arrays in the plain form (scales as 16-bit words) -> the tiled bytes (q8_w4_tile)."""
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    scales = np.ascontiguousarray(scales).view(np.uint16)
    if zeros is not None:
        zeros = np.ascontiguousarray(zeros, dtype=np.uint8)
    K, N, groups = 2 * codes.shape[0], codes.shape[1], scales.shape[0]
    if scales.shape[1] != N or (zeros is not None and zeros.shape != scales.shape) or not groups or K % groups:
        raise ValueError("scales and zeros must be [K / group, N], codes [K / 2, N]")
    flags = (FLAG_W4_ZEROS if zeros is not None else 0) | (FLAG_W4_BF16 if bf16_scales else 0)
    if max(K, N) > _INT_MAX:
        raise ValueError("K and N must be less than 2^31")
    out = np.empty(max(_w4_bytes(K, N, K // groups, flags), 1), dtype=np.uint8)
    _check(lib().q8_w4_tile(codes.ctypes.data, scales.ctypes.data, None if zeros is None else zeros.ctypes.data, K, N,
                            K // groups, flags, out.ctypes.data), "q8_w4_tile")
    return out


def repack4(blocks, K: int, N: int):
    """(codes uint8 [K/2, N], scales float16 [K/32, N]) from N * K/32 Q4_0 checkpoint blocks of 18 bytes (host)."""
    raw = np.frombuffer(bytes(blocks), dtype=np.uint8) if not isinstance(blocks, np.ndarray) else \
        np.ascontiguousarray(blocks).view(np.uint8).reshape(-1)
    if max(abs(K), abs(N)) > _INT_MAX:
        raise ValueError("K and N must be less than 2^31")
    if K > 0 and N > 0 and raw.size != N * (K // Q8_BLOCK) * 18:
        raise ValueError("block buffer size does not match K and N")
    codes = np.empty((max(K // 2, 1), max(N, 1)), dtype=np.uint8)
    scales = np.empty((max(K // Q8_BLOCK, 1), max(N, 1)), dtype=np.float16)
    _check(lib().q8_w4_repack(raw.ctypes.data, K, N, codes.ctypes.data, scales.ctypes.data), "q8_w4_repack")
    return codes, scales


def _x4(x, w):
    """The rows of activation x, checked against weight w."""
    shape = x.shape
    if x.dtype is not w._bf16 or len(shape) != 2 or shape[1] != w.K or x.get_device() != w._index \
            or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous bfloat16 tensor [m, {w.K}] on the weight's device")
    return shape[0]


def _out4(name, t, m, w, dtype, stream):
    """An output [m, Np] of weight w: t, checked, or a new one."""
    if t is None:
        return w._empty((m, w.Np), dtype=dtype, device=w.device) if stream is None else _new((m, w.Np), dtype, w.device, stream)
    if t.dtype is not dtype or tuple(t.shape) != (m, w.Np) or t.get_device() != w._index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor [{m}, {w.Np}] on the weight's device")
    return t


def gemv4(x, w: Weight4, y=None, constant_weights: bool = False, stream=None):
    """y = x . W over a 4-bit weight (q8_gemv4): x bf16 [m, K], 1 <= m <= 512; returns y, fp32 [m, Np] (columns N .. Np-1
    are 0).  constant_weights: as for :func:`gemv`."""
    m = _x4(x, w)
    y = _out4("y", y, m, w, w._f32, stream)
    st = lib().q8_gemv4(x.data_ptr(), w._ref, y.data_ptr(), m, w.K, 1 if constant_weights else 0,
                        _stream_of(stream, w.device))
    if st:
        raise Q8Error(st, "q8_gemv4")
    return y


_POINTERS = [struct.Struct(f"{n}Q") for n in range(9)]


def gemv4_parts(x, weights, ys=None, constant_weights: bool = False, stream=None):
    """Several products of one activation in one call (q8_gemv4_parts); the weights have the same K, group and flags.
    Returns the list of outputs, fp32 [m, Np_p]."""
    n = len(weights)
    if not 1 <= n <= 8:
        raise ValueError("1 to 8 weights")
    if ys is not None and len(ys) != n:
        raise ValueError("an output for each weight")
    w0 = weights[0]
    m, K, index = _x4(x, w0), w0.K, w0._index
    for w in weights:
        if w.K != K or w._index != index:
            raise ValueError("the weights must have the same K and device")
    outs = [_out4("y", None if ys is None else ys[i], m, w, w._f32, stream) for i, w in enumerate(weights)]
    st = lib().q8_gemv4_parts(x.data_ptr(), b"".join([w._packed for w in weights]),
                              _POINTERS[n].pack(*[y.data_ptr() for y in outs]), n, m, K, 1 if constant_weights else 0,
                              _stream_of(stream, w0.device))
    if st:
        raise Q8Error(st, "q8_gemv4_parts")
    return outs


def gemv4_glu(x, gate: Weight4, up: Weight4, out=None, out_bf16=None, want=("f32",), constant_weights: bool = False,
              stream=None):
    """The gated pair (q8_gemv4_glu): silu(x . Wg) * (x . Wu).  ``want``: which outputs to allocate when not given, "f32"
    and/or "bf16" ([m, Np]).  Returns (out, out_bf16), either None when not requested."""
    m = _x4(x, gate)
    if up.K != gate.K or up._index != gate._index:
        raise ValueError("gate and up must have the same K and device")
    if out is not None or "f32" in want:
        out = _out4("out", out, m, gate, gate._f32, stream)
    if out_bf16 is not None or "bf16" in want:
        out_bf16 = _out4("out_bf16", out_bf16, m, gate, gate._bf16, stream)
    st = lib().q8_gemv4_glu(x.data_ptr(), gate._ref, up._ref, None if out is None else out.data_ptr(),
                            None if out_bf16 is None else out_bf16.data_ptr(), m, gate.K, 1 if constant_weights else 0,
                            _stream_of(stream, gate.device))
    if st:
        raise Q8Error(st, "q8_gemv4_glu")
    return out, out_bf16


def gemv4_residual_norm(x, w: Weight4, residual, gamma, eps: float, h=None, out_bf16=None, constant_weights: bool = False,
                        stream=None):
    """A projection, the residual add and the following RMS norm (q8_gemv4_residual_norm): h = residual + x . W, out =
    h / sqrt(mean(h^2) + eps) * gamma.  Returns (h fp32 [m, Np], out bf16 [m, Np]); ``h`` may be ``residual`` (in place)."""
    m = _x4(x, w)
    if residual is None:
        raise ValueError("residual must be given")
    _out4("residual", residual, m, w, w._f32, stream)
    if gamma.dtype is not w._f32 or gamma.numel() < w.N or not gamma.is_contiguous() or gamma.get_device() != w._index:
        raise ValueError("gamma must be a contiguous fp32 tensor of at least N values on the weight's device")
    h = _out4("h", h, m, w, w._f32, stream)
    out_bf16 = _out4("out_bf16", out_bf16, m, w, w._bf16, stream)
    st = lib().q8_gemv4_residual_norm(x.data_ptr(), w._ref, residual.data_ptr(), gamma.data_ptr(), eps, h.data_ptr(),
                                      out_bf16.data_ptr(), m, w.K, 1 if constant_weights else 0,
                                      _stream_of(stream, w.device))
    if st:
        raise Q8Error(st, "q8_gemv4_residual_norm")
    return h, out_bf16


class _Choice(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("repetition", "frequency", "presence", "temperature", "history", "lengths", "prompts",
                                  "bias_ids", "bias", "mask", "mask_rows", "noise")] + \
               [(n, _I) for n in ("history_width", "history_pitch", "history_wide", "bias_width", "mask_count",
                                  "mask_pitch", "noise_pitch")]


_CHOICE = struct.Struct("12Q7i4x")  # the same, packed at a third of the time
assert _CHOICE.size == ctypes.sizeof(_Choice)


def _pitched(name, t, dtype, rows, cols, index):
    """A 2-D tensor's pointer and row pitch: unit column stride, `rows` rows, at least `cols` columns."""
    shape = t.shape
    if t.dtype is dtype and len(shape) == 2 and shape[0] == rows and shape[1] >= cols and t.get_device() == index:
        pitch, unit = t.stride()
        if rows <= 1:
            pitch = shape[1]
        if (unit == 1 or shape[1] == 1) and shape[1] <= pitch <= _INT_MAX and rows <= _INT_MAX:
            return t.data_ptr(), pitch
    raise ValueError(f"{name} must be a 2-D {dtype} CUDA tensor of {rows} rows and at least {cols} columns, unit column stride, "
                     "rows less than 2^31 values apart, on the device of the logits")


def _row_values(name, t, dtype, m, index):
    """The pointer of a value for each row; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.numel() != m or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of {m} values on the logits' device")
    return t.data_ptr()


def choose(logits, N: int | None = None, out=None, repetition=None, frequency=None, presence=None, temperature=None,
           history=None, lengths=None, prompts=None, bias_ids=None, bias=None, mask=None, mask_rows=None, noise=None,
           idx=None, stream=None):
    """Penalties for repeated tokens, biases, temperature and grammar masks on the logits, and the token chosen
    (q8_choose): logits fp32 [m, >= N] (N defaults to the columns).  Returns idx, int64 [m]: the first maximum among the
    allowed tokens, -1 where the mask allows none.

    out: fp32 [m, >= N] that receives the logits after the rules (``logits`` itself: in place; None: not written).
    repetition, frequency, presence, temperature: fp32 [m].  history: int32 or int64 [m, width], of which the first
    ``lengths`` (int32 [m]) tokens of a row count, the first ``prompts`` (int32 [m]) of those as prompt: repetition looks at
    all of them, frequency and presence at the others.  bias_ids int32 and bias fp32 [m, count]: tokens with a bias, ids
    outside the vocabulary are unused places.  mask: int32 [masks, >= ceil(N / 32)], a set bit n % 32 of word n / 32 allows
    token n; mask_rows int32 [m]: the mask of each row, none where it is outside 0 .. masks-1 (default: mask r for row r, of
    which there have to be m).  noise: fp32 [m, >= N], added for the choice where the temperature is above 0 (Gumbel noise
    samples softmax(out))."""
    import torch
    f32, i32 = torch.float32, torch.int32
    index, shape = logits.get_device(), logits.shape
    if index < 0 or len(shape) != 2:
        raise ValueError("logits must be a 2-D CUDA tensor")
    m = shape[0]
    if N is None:
        N = shape[1]
    if N < 1:
        raise ValueError("N must be positive")
    lp, ldl = _pitched("logits", logits, f32, m, N, index)
    op, ldo = (None, 0) if out is None else _pitched("out", out, f32, m, N, index)
    hp = wide = hpitch = hwidth = bp = vp = bwidth = mp = mcount = mpitch = np_ = npitch = 0
    if history is not None:
        if lengths is None:
            raise ValueError("history needs lengths")
        if history.shape[-1]:
            wide = history.dtype is torch.int64
            hp, hpitch = _pitched("history", history, torch.int64 if wide else i32, m, 1, index)
            hwidth = history.shape[1]
    if bias_ids is not None:
        bwidth = bias_ids.shape[-1]
        if bias is None or bias_ids.dtype is not i32 or bias.dtype is not f32 or bias_ids.get_device() != index \
                or bias.get_device() != index or tuple(bias_ids.shape) != (m, bwidth) or bias.shape != bias_ids.shape \
                or not bias_ids.is_contiguous() or not bias.is_contiguous():
            raise ValueError("bias_ids int32 and bias float32 must be contiguous [m, count], on the logits' device")
        if bwidth:
            bp, vp = bias_ids.data_ptr(), bias.data_ptr()
    elif bias is not None:
        raise ValueError("bias needs bias_ids")
    if mask is not None:
        mcount = mask.shape[0]
        if m and mcount < (m if mask_rows is None else 1):
            raise ValueError("a mask for each row, or mask_rows and at least one mask")
        mp, mpitch = _pitched("mask", mask, i32, mcount, (N + 31) // 32, index)
    elif mask_rows is not None:
        raise ValueError("mask_rows needs mask")
    if noise is not None:
        np_, npitch = _pitched("noise", noise, f32, m, N, index)
    if idx is None:
        idx = torch.empty(m, dtype=torch.int64, device=logits.device) if stream is None else \
            _new((m,), torch.int64, logits.device, stream)
    elif idx.dtype is not torch.int64 or idx.numel() != m or not idx.is_contiguous() or idx.get_device() != index:
        raise ValueError("idx must be a contiguous int64 CUDA tensor of m values on the logits' device")
    if m == 0:
        return idx
    c = _CHOICE.pack(_row_values("repetition", repetition, f32, m, index), _row_values("frequency", frequency, f32, m, index),
                     _row_values("presence", presence, f32, m, index), _row_values("temperature", temperature, f32, m, index),
                     hp, _row_values("lengths", lengths, i32, m, index), _row_values("prompts", prompts, i32, m, index), bp,
                     vp, mp, _row_values("mask_rows", mask_rows, i32, m, index), np_, hwidth, hpitch, wide, bwidth, mcount, mpitch, npitch)
    st = lib().q8_choose(lp, ldl, c, op, ldo, idx.data_ptr(), m, N, _stream_of(stream, logits.device))
    if st:
        raise Q8Error(st, "q8_choose")
    return idx


def residual_norm_launches() -> int:
    """Kernel launches one gemv_residual_norm call makes, by the library's current rule: the product, then the norm as
    a launch of its own (2); 1 when the one-launch fold is selected (tuning ``norm_fold`` = 1)."""
    return 1 if get_tuning("norm_fold") == 1 else 2


def device_fault(clear: bool = False) -> int:
    """The device fault word (nonzero when a kernel's bounded pipeline wait ran out); see q8_device_fault."""
    word = ctypes.c_uint(0)
    _check(lib().q8_device_fault(ctypes.byref(word), int(clear)), "q8_device_fault")
    return word.value


def repack(blocks, K: int, N: int, scale: str = "f32"):
    """(q int8 [K, Np], s fp32 [K/32, Np]) from N * K/32 checkpoint blocks (host): 36-byte blocks with an fp32 scale
    (q8_repack), or with scale="f16" GGML-style 34-byte blocks with a binary16 scale (q8_repack_f16)."""
    size = {"f32": 36, "f16": 34}[scale]
    raw = np.frombuffer(bytes(blocks), dtype=np.uint8) if not isinstance(blocks, np.ndarray) else \
        np.ascontiguousarray(blocks).view(np.uint8).reshape(-1)
    Np = padded_n(N) if N > 0 else 1
    nb = max(K // Q8_BLOCK, 1)
    if K > 0 and N > 0 and raw.size != N * nb * size:
        raise ValueError("block buffer size does not match K and N")
    q = np.empty((max(K, 1), Np), dtype=np.int8)
    s = np.empty((nb, Np), dtype=np.float32)
    fn = lib().q8_repack if scale == "f32" else lib().q8_repack_f16
    name = "q8_repack" if scale == "f32" else "q8_repack_f16"
    _check(fn(raw.ctypes.data, K, N, q.ctypes.data, s.ctypes.data), name)
    return q, s


def quantize(w):
    """(q int8 [K, Np], s fp32 [K/32, Np]) for a declared fp64 weight [K, N] (host); raises Q8Error if not Q8_0."""
    w = np.ascontiguousarray(w, dtype=np.float64)
    K, N = w.shape
    Np = padded_n(N) if N > 0 else 1
    q = np.empty((max(K, 1), Np), dtype=np.int8)
    s = np.empty((max(K // Q8_BLOCK, 1), Np), dtype=np.float32)
    _check(lib().q8_quantize(w.ctypes.data, K, N, q.ctypes.data, s.ctypes.data), "q8_quantize")
    return q, s
