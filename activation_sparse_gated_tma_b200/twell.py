"""Python binding of libtwell.so (include/twell.h): argument marshalling only.

Every step of the forward path runs in the library's CUDA kernels; PyTorch
provides device memory and the current stream.  There is no fallback: if the
library is missing or the device is not an sm_100 GPU, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Dict, NamedTuple, Optional, Tuple

import torch

from . import build as _build

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtwell.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "twell.h")

OK, ERR_INVALID, ERR_CAPACITY, ERR_CUDA, ERR_DEVICE_CHECK, ERR_UNSUPPORTED = range(6)


class TwellError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {message} (status {status})")
        self.status = status


class CapacityError(TwellError):
    def __init__(self, status, where, message, n_over):
        super().__init__(status, where, message)
        self.n_over = n_over


class _TwellBuf(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("counts", "idx", "vals", "dense_rows", "row_slot", "slot_row", "ctrl", "x_over", "h_over",
                 "units", "z")] + \
               [(n, ctypes.c_int) for n in ("M", "K", "N", "T", "C", "R_cap")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libtwell.so (building it first if sources are newer and nvcc exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH) or (_build.needs_build() and os.path.exists(_build.NVCC)):
        _build.build()
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m activation_sparse_gated_tma_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    LL, F = ctypes.c_longlong, ctypes.c_float
    IP = ctypes.POINTER(ctypes.c_int)
    BP = ctypes.POINTER(_TwellBuf)
    sig = {
        "twell_buf_bytes": (S, [I, I, I, I, I, I]),
        "twell_buf_init": (I, [BP, P, S, I, I, I, I, I, I]),
        "twell_gate_pack": (I, [P, P, I, I, I, BP, IP, P]),
        "twell_ffn_fwd": (I, [P, P, P, BP, I, P, P]),
        "twell_ffn_fused": (I, [P, P, P, P, I, I, I, BP, P, IP, P]),
        "twell_bwd_scratch_bytes": (S, [I, I, I, I, I, I]),
        "twell_ffn_bwd": (I, [P, P, P, P, BP, P, I, P, P, P, P, P, S, P]),
        "twell_bwd_slot_route": (I, [I]),
        "twell_read_status": (I, [BP, IP, IP, P]),
        "twell_layer_norm_fwd": (I, [P, I, LL, P, P, I, I, I, F, P, I, LL, P, P, P]),
        "twell_layer_norm_int8": (I, [P, I, LL, P, P, I, I, I, F, P, LL, P, P, P, P]),
        "twell_layer_norm_bwd_scratch_bytes": (S, [I, I]),
        "twell_layer_norm_bwd": (I, [P, I, LL, P, I, LL, P, P, P, I, I, I, P, LL, P, P, P, S, P]),
        "twell_quantize_rows": (I, [P, I, LL, I, I, P, LL, P, P]),
        "twell_dequantize_rows": (I, [P, LL, P, I, I, P, I, LL, P]),
        "twell_int8_linear": (I, [P, LL, P, P, LL, P, P, I, I, I, P, I, LL, P]),
        "twell_int8_gated": (I, [P, LL, P, P, LL, P, P, LL, P, I, I, I, P, I, LL, P]),
        "twell_int8_cut": (I, [I, I]),
        "dense_ffn_fwd": (I, [P, P, P, P, I, I, I, P, P, P]),
        "dense_ffn_fwd_bf16h": (I, [P, P, P, P, I, I, I, P, P, P]),
        "dense_ffn_fwd_noalloc": (I, [P, P, P, P, I, I, I, P, P]),
        "twell_test_expire_wait": (I, [ctypes.c_longlong]),
        "twell_status_str": (ctypes.c_char_p, [I]),
        "twell_last_error": (ctypes.c_char_p, []),
        "twell_last_launch_count": (I, []),
        "twell_trace_events": (I, [P, I]),
        "twell_trace_count": (I, []),
        "twell_trace_name": (ctypes.c_char_p, [I]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


def header_functions() -> list:
    """Names of the functions include/twell.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b((?:twell|dense)_\w+)\s*\(", text)))


def _check(status: int, where: str):
    if status != OK:
        L = lib()
        msg = (L.twell_last_error() or b"").decode() or L.twell_status_str(status).decode()
        raise TwellError(status, where, msg)


def last_launch_count() -> int:
    return lib().twell_last_launch_count()


class KernelTrace:
    """Brackets every kernel the library launches (on this thread) with CUDA
    events, for per-kernel device times of live runs.

        with KernelTrace(capacity=16) as tr:
            ...library calls...
        torch.cuda.synchronize(); tr.times_ms() -> [(kernel name, ms), ...]
    """

    def __init__(self, capacity: int = 16):
        self.capacity = capacity
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * capacity)]
        for e in self.events:      # torch creates the CUDA event lazily, on first record
            e.record()
        self._arr = (ctypes.c_void_p * (2 * capacity))(*[e.cuda_event for e in self.events])
        self.count = 0
        self.names = []

    def __enter__(self):
        _check(lib().twell_trace_events(self._arr, self.capacity), "twell_trace_events")
        return self

    def __exit__(self, *exc):
        L = lib()
        self.count = L.twell_trace_count()
        self.names = [L.twell_trace_name(i).decode() for i in range(self.count)]
        L.twell_trace_events(None, 0)
        return False

    def times_ms(self):
        return [(self.names[i], self.events[2 * i].elapsed_time(self.events[2 * i + 1])) for i in range(self.count)]


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _bf16(t: torch.Tensor, name: str, shape) -> int:
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


class TwellBuffers:
    """TwELL activations + dense-row backup in one device allocation.

    Views (torch tensors over the same memory): counts [M][N/T] uint16 (as
    int16), idx [M][N/T][C] uint8, vals [M][N/T][C] float32, dense_rows
    [R_cap][N] float32, row_slot [M] int32, slot_row [R_cap] int32, ctrl [64] int32.
    """

    def __init__(self, M: int, K: int, N: int, T: int, C: int, R_cap: Optional[int] = None, device=None):
        L = lib()
        R_cap = R_cap if R_cap is not None else max(1, -(-M // 8))
        nbytes = L.twell_buf_bytes(M, K, N, T, C, R_cap)
        if nbytes == 0:
            raise ValueError(f"unsupported TwELL sizes M={M} K={K} N={N} T={T} C={C} R_cap={R_cap}")
        device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.storage = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        base = self.storage.data_ptr()
        self._off0 = (-base) % 256
        self.buf = _TwellBuf()
        _check(L.twell_buf_init(ctypes.byref(self.buf), base + self._off0, nbytes, M, K, N, T, C, R_cap),
               "twell_buf_init")
        self.M, self.K, self.N, self.T, self.C, self.R_cap = M, K, N, T, C, R_cap
        self.n_over_known: Optional[int] = None

    def _view(self, field: str, dtype, shape):
        off = getattr(self.buf, field) - self.storage.data_ptr()
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.storage[off:off + nbytes].view(dtype).view(*shape)

    @property
    def counts(self):
        return self._view("counts", torch.int16, (self.M, self.N // self.T))

    @property
    def idx(self):
        return self._view("idx", torch.uint8, (self.M, self.N // self.T, self.C))

    @property
    def vals(self):
        return self._view("vals", torch.float32, (self.M, self.N // self.T, self.C))

    @property
    def dense_rows(self):
        return self._view("dense_rows", torch.float32, (self.R_cap, self.N))

    @property
    def row_slot(self):
        return self._view("row_slot", torch.int32, (self.M,))

    @property
    def slot_row(self):
        return self._view("slot_row", torch.int32, (self.R_cap,))

    @property
    def ctrl(self):
        return self._view("ctrl", torch.int32, (64,))

    def to_host(self) -> Dict[str, "object"]:
        """Copy the TwELL arrays to host numpy (counts as uint16)."""
        import numpy as np
        return {
            "counts": self.counts.cpu().numpy().view(np.uint16),
            "idx": self.idx.cpu().numpy(),
            "vals": self.vals.cpu().numpy(),
            "dense_rows": self.dense_rows.cpu().numpy(),
            "row_slot": self.row_slot.cpu().numpy(),
            "slot_row": self.slot_row.cpu().numpy(),
            "ctrl": self.ctrl.cpu().numpy(),
        }


def gate_pack(x: torch.Tensor, wg_t: torch.Tensor, tw: TwellBuffers, sync: bool = False, stream=None) -> Optional[int]:
    """twell_gate_pack.  With sync=True returns n_over and raises CapacityError when > R_cap."""
    M, K = x.shape
    N = wg_t.shape[0]
    px = _bf16(x, "x", (M, K))
    pw = _bf16(wg_t, "wg_t", (N, K))
    L = lib()
    n_over = ctypes.c_int(-1)
    st = L.twell_gate_pack(px, pw, M, K, N, ctypes.byref(tw.buf), ctypes.byref(n_over) if sync else None,
                           _stream(stream))
    if st == ERR_CAPACITY:
        raise CapacityError(st, "twell_gate_pack", (L.twell_last_error() or b"").decode(), n_over.value)
    _check(st, "twell_gate_pack")
    tw.n_over_known = n_over.value if sync else None
    return n_over.value if sync else None


def ffn_fwd(x: torch.Tensor, wu_t: torch.Tensor, wd: torch.Tensor, tw: TwellBuffers,
            y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """twell_ffn_fwd: y [M][K] fp32 from TwELL (fused sparse up+down, then the dense-row path)."""
    M, K = x.shape
    N = wu_t.shape[0]
    if y is None:
        y = torch.empty((M, K), dtype=torch.float32, device=x.device)
    if y.dtype != torch.float32 or not y.is_contiguous() or tuple(y.shape) != (M, K):
        raise ValueError("y must be a contiguous float32 tensor of shape (M, K)")
    st = lib().twell_ffn_fwd(_bf16(x, "x", (M, K)), _bf16(wu_t, "wu_t", (N, K)), _bf16(wd, "wd", (N, K)),
                             ctypes.byref(tw.buf), K, y.data_ptr(), _stream(stream))
    _check(st, "twell_ffn_fwd")
    return y


def ffn_fused(x: torch.Tensor, wg_t: torch.Tensor, wu_t: torch.Tensor, wd: torch.Tensor, tw: TwellBuffers,
              y: Optional[torch.Tensor] = None, sync: bool = False, stream=None) -> torch.Tensor:
    """twell_ffn_fused: the whole sparse forward in one call (one persistent
    kernel after the reset for M <= TWELL_SMALL_M).  With sync=True raises
    CapacityError when the dense-row slots ran out."""
    M, K = x.shape
    N = wg_t.shape[0]
    if y is None:
        y = torch.empty((M, K), dtype=torch.float32, device=x.device)
    if y.dtype != torch.float32 or not y.is_contiguous() or tuple(y.shape) != (M, K):
        raise ValueError("y must be a contiguous float32 tensor of shape (M, K)")
    L = lib()
    n_over = ctypes.c_int(-1)
    st = L.twell_ffn_fused(_bf16(x, "x", (M, K)), _bf16(wg_t, "wg_t", (N, K)), _bf16(wu_t, "wu_t", (N, K)),
                           _bf16(wd, "wd", (N, K)), M, K, N, ctypes.byref(tw.buf), y.data_ptr(),
                           ctypes.byref(n_over) if sync else None, _stream(stream))
    if st == ERR_CAPACITY:
        raise CapacityError(st, "twell_ffn_fused", (L.twell_last_error() or b"").decode(), n_over.value)
    _check(st, "twell_ffn_fused")
    tw.n_over_known = n_over.value if sync else None
    return y


def ffn_bwd(x: torch.Tensor, wg_t: torch.Tensor, wu_t: torch.Tensor, wd: torch.Tensor, tw: TwellBuffers,
            dy: torch.Tensor, scratch: Optional[torch.Tensor] = None, stream=None):
    """twell_ffn_bwd: (dx, dwg_t, dwu_t, dwd), all fp32, from the forward's TwELL
    buffer `tw` and the upstream gradient dy [M][K] fp32."""
    M, K = x.shape
    N = wg_t.shape[0]
    if dy.dtype != torch.float32 or not dy.is_contiguous() or tuple(dy.shape) != (M, K):
        raise ValueError("dy must be a contiguous float32 tensor of shape (M, K)")
    L = lib()
    need = L.twell_bwd_scratch_bytes(M, K, N, tw.T, tw.C, tw.R_cap)
    if need == 0:
        raise ValueError("invalid sizes for twell_ffn_bwd")
    if scratch is None or scratch.numel() < need:
        scratch = torch.empty(need, dtype=torch.uint8, device=x.device)
    dx = torch.empty((M, K), dtype=torch.float32, device=x.device)
    dg, du, dd = (torch.empty((N, K), dtype=torch.float32, device=x.device) for _ in range(3))
    st = L.twell_ffn_bwd(_bf16(x, "x", (M, K)), _bf16(wg_t, "wg_t", (N, K)), _bf16(wu_t, "wu_t", (N, K)),
                         _bf16(wd, "wd", (N, K)), ctypes.byref(tw.buf), dy.data_ptr(), K, dx.data_ptr(),
                         dg.data_ptr(), du.data_ptr(), dd.data_ptr(), scratch.data_ptr(), scratch.numel(),
                         _stream(stream))
    _check(st, "twell_ffn_bwd")
    return dx, dg, du, dd


def read_status(tw: TwellBuffers, stream=None):
    """Synchronise and return (status, n_over, device_flags)."""
    n = ctypes.c_int(0)
    f = ctypes.c_int(0)
    st = lib().twell_read_status(ctypes.byref(tw.buf), ctypes.byref(n), ctypes.byref(f), _stream(stream))
    return st, n.value, f.value


def dense_ffn(x: torch.Tensor, wg_t: torch.Tensor, wu_t: torch.Tensor, wd: torch.Tensor,
              h_scratch: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, stream=None,
              bf16_h: bool = False) -> torch.Tensor:
    """dense_ffn_fwd: the same y with dense tensor-core GEMMs.

    h is materialised as bf16 hi + lo halves (h_scratch [M][2N]); with
    bf16_h=True, dense_ffn_fwd_bf16h keeps it as one bf16 (h_scratch [M][N]).
    """
    M, K = x.shape
    N = wg_t.shape[0]
    hcols = N if bf16_h else 2 * N
    if h_scratch is None:
        h_scratch = torch.empty((M, hcols), dtype=torch.bfloat16, device=x.device)
    if y is None:
        y = torch.empty((M, K), dtype=torch.float32, device=x.device)
    if y.dtype != torch.float32 or not y.is_contiguous() or tuple(y.shape) != (M, K):
        raise ValueError("y must be a contiguous float32 tensor of shape (M, K)")
    f = lib().dense_ffn_fwd_bf16h if bf16_h else lib().dense_ffn_fwd
    st = f(_bf16(x, "x", (M, K)), _bf16(wg_t, "wg_t", (N, K)), _bf16(wu_t, "wu_t", (N, K)),
           _bf16(wd, "wd", (N, K)), M, K, N, _bf16(h_scratch, "h_scratch", (M, hcols)), y.data_ptr(),
           _stream(stream))
    _check(st, "dense_ffn_fwd_bf16h" if bf16_h else "dense_ffn_fwd")
    return y


def dense_ffn_noalloc(x: torch.Tensor, wg_t: torch.Tensor, wu_t: torch.Tensor, wd: torch.Tensor,
                      y: torch.Tensor, stream=None) -> torch.Tensor:
    """dense_ffn_fwd_noalloc: dense_ffn with h in the library's fixed device array."""
    M, K = x.shape
    N = wg_t.shape[0]
    if y.dtype != torch.float32 or not y.is_contiguous() or tuple(y.shape) != (M, K) or not y.is_cuda:
        raise ValueError("y must be a contiguous CUDA float32 tensor of shape (M, K)")
    st = lib().dense_ffn_fwd_noalloc(_bf16(x, "x", (M, K)), _bf16(wg_t, "wg_t", (N, K)),
                                     _bf16(wu_t, "wu_t", (N, K)), _bf16(wd, "wd", (N, K)), M, K, N,
                                     y.data_ptr(), _stream(stream))
    _check(st, "dense_ffn_fwd_noalloc")
    return y


# ---------------------------------------------------------------------------
# Rows of activations: layer norm, its backward pass, int8 rows and products.

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.int8: 3}  # twell_dtype
_FLOATING = (torch.float32, torch.bfloat16, torch.float16)
_I8 = (torch.int8,)
_INT_MAX = 2 ** 31 - 1  # sizes are C ints


def _elsewhere(stream, *tensors) -> bool:
    """Whether a call on `tensors` (on one CUDA device) has to change the
    current device or stream first; small calls are bound by the host, so the
    usual case does neither."""
    d = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != d:
            raise ValueError(f"tensors on {tensors[0].device} and {t.device}")
    if d < 0:
        raise ValueError(f"tensors must be on a CUDA device, not {tensors[0].device}")
    return stream is not None or d != _current_device()


def _there(stream, t: torch.Tensor):
    """Context of such a call: the tensors' device made current, and a given
    stream too, so that what the call allocates belongs to the stream it runs on."""
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError(f"stream on {stream.device}, tensors on {t.device}")
    return torch.cuda.stream(stream)


def _current_device() -> int:
    return torch._C._cuda_getDevice()  # torch.cuda.current_device() less its lazy initialisation: t is on a device


def _here(t: torch.Tensor) -> int:
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _rows(t: torch.Tensor, name: str, dtypes, shape=None) -> int:
    """Row stride of a matrix argument (rows may be strided, elements not)."""
    size = t.shape
    if len(size) != 2 or t.dtype not in dtypes or (shape is not None and size != shape):
        raise ValueError(f"{name} must be a matrix{'' if shape is None else f' of shape {tuple(shape)}'} of "
                         f"{' or '.join(map(str, dtypes))}, got {t.dtype} {tuple(size)}")
    rows, cols = size
    if rows > _INT_MAX or cols > _INT_MAX:  # ctypes would cut them to 32 bits
        raise ValueError(f"{name} must have at most {_INT_MAX} rows and columns, got {tuple(size)}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name}'s elements of a row must be contiguous (strides {t.stride()})")
    if rows <= 1:  # the stride of a single row says nothing
        return -(-cols // 16) * 16
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap (strides {t.stride()})")
    return ld


def _vector(t: Optional[torch.Tensor], name: str, n: int, dtypes=(torch.float32,)) -> Optional[int]:
    if t is None:
        return None
    if t.dtype not in dtypes or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} {' or '.join(map(str, dtypes))}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _affine(weight, bias, D):
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError(f"weight and bias must have one type, got {weight.dtype} and {bias.dtype}")
    ref = weight if weight is not None else bias
    return (_vector(weight, "weight", D, _FLOATING), _vector(bias, "bias", D, _FLOATING),
            0 if ref is None else _DTYPES[ref.dtype])


def _matrix(M: int, N: int, dtype, like: torch.Tensor) -> torch.Tensor:
    return like.new_empty((M, N), dtype=dtype)


def _rows_like(x: torch.Tensor, dtype) -> torch.Tensor:
    """Contiguous, of x's shape (empty_like takes half a microsecond less than new_empty)."""
    return torch.empty_like(x) if dtype is x.dtype and x.is_contiguous() else x.new_empty(x.shape, dtype=dtype)


def _two_vectors(n: int, like: torch.Tensor):
    a = like.new_empty(n, dtype=torch.float32)
    return a, torch.empty_like(a)


def _int8_rows(M: int, K: int, like: torch.Tensor):
    """int8 [M][K] whose row stride is a multiple of 16, as the products need it."""
    ld = -(-K // 16) * 16
    if ld == K:
        return _matrix(M, K, torch.int8, like), ld
    return like.new_empty_strided((M, K), (ld, 1), dtype=torch.int8), ld


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
               stats: bool = False, stream=None):
    """twell_layer_norm_fwd: y = (x - mean) rstd weight + bias over the rows of x [M][D].

    out_dtype (default x's) is x's type, float32, or any of the three when x is
    float32; `out` gives the output, whose rows may be strided.  With
    stats=True returns (y, mean, rstd), what layer_norm_bwd needs."""
    ldx = _rows(x, "x", _FLOATING)
    M, D = x.shape
    w, b, wt = _affine(weight, bias, D)
    if out is not None:
        if out_dtype not in (None, out.dtype):
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
        ldy = _rows(out, "out", _FLOATING, (M, D))
    elif out_dtype is not None and out_dtype not in _FLOATING:
        raise ValueError(f"out_dtype must be one of {_FLOATING}, got {out_dtype}")
    if _elsewhere(stream, x, weight, bias, out):
        with _there(stream, x):
            return layer_norm(x, weight, bias, eps, out, out_dtype, stats)
    if out is None:
        out, ldy = _rows_like(x, out_dtype or x.dtype), D
    mean = rstd = pm = pr = None
    if stats:
        mean, rstd = _two_vectors(M, x)
        pm, pr = mean.data_ptr(), rstd.data_ptr()
    _check(lib().twell_layer_norm_fwd(x.data_ptr(), _DTYPES[x.dtype], ldx, w, b, wt, M, D, eps, out.data_ptr(),
                                      _DTYPES[out.dtype], ldy, pm, pr, _here(x)), "twell_layer_norm_fwd")
    return (out, mean, rstd) if stats else out


def layer_norm_int8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                    eps: float = 1e-5, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """twell_layer_norm_int8: the norm of x's rows as int8 rows and their scales,
    (q [M][D], scale [M]), ready for int8_linear and int8_gated."""
    ldx = _rows(x, "x", _FLOATING)
    M, D = x.shape
    w, b, wt = _affine(weight, bias, D)
    if _elsewhere(stream, x, weight, bias):
        with _there(stream, x):
            return layer_norm_int8(x, weight, bias, eps)
    q, ldq = _int8_rows(M, D, x)
    scale = x.new_empty(M, dtype=torch.float32)
    _check(lib().twell_layer_norm_int8(x.data_ptr(), _DTYPES[x.dtype], ldx, w, b, wt, M, D, eps, q.data_ptr(), ldq,
                                       scale.data_ptr(), None, None, _here(x)), "twell_layer_norm_int8")
    return q, scale


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: Optional[torch.Tensor] = None, param_grads: bool = True,
                   scratch: Optional[torch.Tensor] = None, stream=None):
    """twell_layer_norm_bwd: (dx, dweight, dbias) from the forward's input, mean
    and rstd and the upstream gradient dy (x's type, float32, or any of the
    three when x is float32).  dx is of x's type, the parameters' gradients are
    float32 (None with param_grads=False)."""
    ldx = _rows(x, "x", _FLOATING)
    M, D = x.shape
    lddy = _rows(dy, "dy", _FLOATING, (M, D))
    w = _vector(weight, "weight", D, _FLOATING)
    pm, pr = _vector(mean, "mean", M), _vector(rstd, "rstd", M)
    if scratch is not None and not scratch.is_contiguous():
        raise ValueError("scratch must be contiguous")
    if _elsewhere(stream, x, dy, mean, rstd, weight, scratch):
        with _there(stream, x):
            return layer_norm_bwd(dy, x, mean, rstd, weight, param_grads, scratch)
    L = lib()
    dx = _rows_like(x, x.dtype)
    dw = db = pw = pb = ps = None
    size = 0
    if param_grads:
        dw, db = _two_vectors(D, x)
        pw, pb = dw.data_ptr(), db.data_ptr()
        if scratch is None:
            size = L.twell_layer_norm_bwd_scratch_bytes(M, D)
            scratch = dw.new_empty(size // 4)
        else:
            size = scratch.numel() * scratch.element_size()
        ps = scratch.data_ptr()
    _check(L.twell_layer_norm_bwd(dy.data_ptr(), _DTYPES[dy.dtype], lddy, x.data_ptr(), _DTYPES[x.dtype], ldx, pm, pr, w,
                                  0 if weight is None else _DTYPES[weight.dtype], M, D, dx.data_ptr(), D, pw, pb, ps,
                                  size, _here(x)), "twell_layer_norm_bwd")
    return dx, dw, db


def quantize_rows(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """twell_quantize_rows: (q int8 [M][K], scale [M]) with x ~ q scale; for
    activations (a scale per token) and weights [N][K] (one per channel)."""
    ldx = _rows(x, "x", _FLOATING)
    M, K = x.shape
    if _elsewhere(stream, x):
        with _there(stream, x):
            return quantize_rows(x)
    q, ldq = _int8_rows(M, K, x)
    scale = x.new_empty(M, dtype=torch.float32)
    _check(lib().twell_quantize_rows(x.data_ptr(), _DTYPES[x.dtype], ldx, M, K, q.data_ptr(), ldq, scale.data_ptr(),
                                     _here(x)), "twell_quantize_rows")
    return q, scale


def dequantize_rows(q: torch.Tensor, scale: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                    stream=None) -> torch.Tensor:
    """twell_dequantize_rows: q scale, of out_dtype."""
    ldq = _rows(q, "q", _I8)
    M, K = q.shape
    ps = _vector(scale, "scale", M)
    if out_dtype not in _FLOATING:
        raise ValueError(f"out_dtype must be one of {_FLOATING}, got {out_dtype}")
    if _elsewhere(stream, q, scale):
        with _there(stream, q):
            return dequantize_rows(q, scale, out_dtype)
    y = _matrix(M, K, out_dtype, q)
    _check(lib().twell_dequantize_rows(q.data_ptr(), ldq, ps, M, K, y.data_ptr(), _DTYPES[out_dtype], K, _here(q)),
           "twell_dequantize_rows")
    return y


def _product_rows(x, w, name):
    """Row strides and sizes of a product's int8 operands."""
    ldx, ldw = _rows(x, "x", _I8), _rows(w, name, _I8)
    (M, K), (N, Kw) = x.shape, w.shape
    if Kw != K:
        raise ValueError(f"x {tuple(x.shape)} and {name} {tuple(w.shape)} must have rows of one length")
    return ldx, ldw, M, N, K


def _product_out(out, out_dtype, M, N):
    if out is not None:
        return _rows(out, "out", _FLOATING, (M, N))
    if out_dtype not in _FLOATING:
        raise ValueError(f"out_dtype must be one of {_FLOATING}, got {out_dtype}")
    return N


def int8_linear(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """twell_int8_linear: y [M][N] = x w^T x_scale w_scale (+ bias) from int8
    rows x [M][K] and w [N][K] (bases 16-byte aligned, row strides multiples of
    16, as quantize_rows makes them)."""
    ldx, ldw, M, N, K = _product_rows(x, w, "w")
    ldy = _product_out(out, out_dtype, M, N)
    xs, ws, pb = _vector(x_scale, "x_scale", M), _vector(w_scale, "w_scale", N), _vector(bias, "bias", N)
    if _elsewhere(stream, x, x_scale, w, w_scale, bias, out):
        with _there(stream, x):
            return int8_linear(x, x_scale, w, w_scale, bias, out_dtype, out)
    y = _matrix(M, N, out_dtype, x) if out is None else out
    _check(lib().twell_int8_linear(x.data_ptr(), ldx, xs, w.data_ptr(), ldw, ws, pb, M, N, K, y.data_ptr(),
                                   _DTYPES[y.dtype], ldy, _here(x)), "twell_int8_linear")
    return y


def int8_gated(x: torch.Tensor, x_scale: torch.Tensor, wg: torch.Tensor, wg_scale: torch.Tensor, wu: torch.Tensor,
               wu_scale: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """twell_int8_gated: h [M][N] = u ReLU(g) with g, u the int8 products of x
    with wg and wu (operands as for int8_linear)."""
    ldx, ldg, M, N, K = _product_rows(x, wg, "wg")
    ldu = _rows(wu, "wu", _I8, (N, K))
    ldh = _product_out(out, out_dtype, M, N)
    xs, gs, us = _vector(x_scale, "x_scale", M), _vector(wg_scale, "wg_scale", N), _vector(wu_scale, "wu_scale", N)
    if _elsewhere(stream, x, x_scale, wg, wg_scale, wu, wu_scale, out):
        with _there(stream, x):
            return int8_gated(x, x_scale, wg, wg_scale, wu, wu_scale, out_dtype, out)
    h = _matrix(M, N, out_dtype, x) if out is None else out
    _check(lib().twell_int8_gated(x.data_ptr(), ldx, xs, wg.data_ptr(), ldg, gs, wu.data_ptr(), ldu, us, M, N, K,
                                  h.data_ptr(), _DTYPES[h.dtype], ldh, _here(x)), "twell_int8_gated")
    return h


def int8_cut(token_tile: int = 0, k_splits: int = 1) -> None:
    """twell_int8_cut: how the following int8 products on this thread are cut;
    0 chooses by estimated time, 256 CTA pairs, 16 to 128 tiles of that many
    tokens with a reduction of k_splits shares (per thread)."""
    _check(lib().twell_int8_cut(int(token_tile), int(k_splits)), "twell_int8_cut")


class Int8FFN(NamedTuple):
    """The dense FFN's weights as int8 rows with a scale per output channel:
    wg, wu [N][K] as in the bf16 layout, wd transposed to [K][N] (each output
    column of y is one row)."""
    wg: torch.Tensor
    wg_scale: torch.Tensor
    wu: torch.Tensor
    wu_scale: torch.Tensor
    wd_t: torch.Tensor
    wd_scale: torch.Tensor


def int8_ffn_weights(wg_t: torch.Tensor, wu_t: torch.Tensor, wd: torch.Tensor) -> Int8FFN:
    """Quantise the FFN's weights (all [N][K]) once, for dense_ffn_int8."""
    return Int8FFN(*quantize_rows(wg_t), *quantize_rows(wu_t), *quantize_rows(wd.t().contiguous()))


def dense_ffn_int8(x: torch.Tensor, weights: Int8FFN, norm=None, out_dtype: torch.dtype = torch.float32,
                   stream=None, h_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The dense FFN (dense_ffn) in 8-bit integers: x's rows quantised, the
    gated pair of products, h's rows quantised, the down product.  norm =
    (weight, bias, eps) applies the layer norm to x first (layer_norm_int8).

    h is held in h_dtype between its product and its quantisation: bfloat16
    halves the bytes, and its half step of 2^-9 to 2^-8 of a value stays below
    the int8 half step of 1/254 of the row's largest; with float32 h is rounded
    once, to int8 (float16 rows may pass that type's range)."""
    q, s = quantize_rows(x, stream) if norm is None else layer_norm_int8(x, *norm, stream=stream)
    h = int8_gated(q, s, weights.wg, weights.wg_scale, weights.wu, weights.wu_scale, out_dtype=h_dtype, stream=stream)
    q, s = quantize_rows(h, stream)
    return int8_linear(q, s, weights.wd_t, weights.wd_scale, out_dtype=out_dtype, stream=stream)


def bwd_slot_route(route: int) -> None:
    """twell_bwd_slot_route: 0 chooses the slotted rows' backward route by
    their entry count, 1 forces the dense-slot GEMMs, 2 the gather passes
    (for the calling thread)."""
    _check(lib().twell_bwd_slot_route(int(route)), "twell_bwd_slot_route")


def test_expire_wait(limit_ns: int) -> None:
    """twell_test_expire_wait: arm a one-shot expiring device wait for the next
    ffn_fwd (large batches) or ffn_fused (small batches)."""
    _check(lib().twell_test_expire_wait(int(limit_ns)), "twell_test_expire_wait")


def sparse_ffn(x: torch.Tensor, wg_t: torch.Tensor, wu_t: torch.Tensor, wd: torch.Tensor, T: int, C: int,
               tw: Optional[TwellBuffers] = None, y: Optional[torch.Tensor] = None, sync: bool = True, norm=None):
    """Whole sparse forward: gate_pack (+ one retry with a larger dense-row buffer
    on capacity overflow, when sync) then ffn_fwd.  Returns (y, tw).

    norm = (weight, bias, eps) applies the layer norm to x first: x may then be
    float32 or bfloat16, and the FFN runs on its bfloat16 output.  (A weight of
    0 and a bias of 1 in the last column make it the gate's bias column.)"""
    M, K = x.shape
    if norm is not None:
        x = layer_norm(x, *norm, out_dtype=torch.bfloat16)
    N = wg_t.shape[0]
    if tw is None:
        tw = TwellBuffers(M, K, N, T, C, device=x.device)
    try:
        gate_pack(x, wg_t, tw, sync=sync)
    except CapacityError as e:
        tw = TwellBuffers(M, K, N, T, C, R_cap=e.n_over, device=x.device)
        gate_pack(x, wg_t, tw, sync=True)
    return ffn_fwd(x, wu_t, wd, tw, y), tw
