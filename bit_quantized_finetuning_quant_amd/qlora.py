"""ctypes binding of the gfx950 QLoRA library (``libqlora_gfx950.so``).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/qlora.h``.  PyTorch supplies
device memory (``data_ptr()``) and the stream (``cuda_stream``).  There is no
fallback: if the library is missing, every call raises.
"""

import ctypes
import functools
import os
import threading
from contextlib import nullcontext
from dataclasses import dataclass
from typing import NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqlora_gfx950.so")

QLORA_F32, QLORA_BF16 = 0, 1
QLORA_NF4_FP32_CONSTANTS = 1
STATUS_NAMES = {0: "QLORA_OK", 1: "QLORA_ERR_NULL", 2: "QLORA_ERR_SHAPE", 3: "QLORA_ERR_ALIGN",
                4: "QLORA_ERR_WORKSPACE", 5: "QLORA_ERR_DTYPE", 6: "QLORA_ERR_HIP",
                7: "QLORA_ERR_NONFINITE", 8: "QLORA_ERR_VALUE", 9: "QLORA_ERR_MEMORY", 10: "QLORA_ERR_SCRATCH"}


class QloraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class NF4WeightStruct(ctypes.Structure):
    _fields_ = [("n_out", ctypes.c_int64), ("n_in", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("absmax_fp8", ctypes.c_void_p), ("absmax_scale", ctypes.c_void_p),
                ("absmax_mean", ctypes.c_void_p), ("flags", ctypes.c_uint32)]


class Act8Struct(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("K", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "qlora_nf4_sizes": (ctypes.c_int, [_I64, _I64, _P, _P, _P]),
    "qlora_nf4_bytes": (_SZ, [_I64, _I64]),
    "qlora_nf4_bytes_flags": (_SZ, [_I64, _I64, ctypes.c_uint32]),
    "qlora_quantize_workspace_bytes": (_SZ, [_I64, _I64]),
    "qlora_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64, ctypes.c_int]),
    "qlora_nf4_codebook": (None, [_P]),
    "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_version": (ctypes.c_char_p, []),
    "qlora_quantize": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _SZ, _P]),
    "qlora_dequantize": (ctypes.c_int, [_P, _P, _P]),
    "qlora_dequantize_many": (ctypes.c_int, [_P, ctypes.c_int, _P, _P]),
    "qlora_linear_fwd": (ctypes.c_int, [_P, _I64, _P, _P, _P, ctypes.c_int, ctypes.c_float, _P, _P, _P, _SZ, _P]),
    "qlora_linear_bwd": (ctypes.c_int, [_P, _P, _I64, _P, _P, _P, ctypes.c_int, ctypes.c_float, _P, _P, _P, _P,
                                        _P, _SZ, _P]),
    "qlora_linear_fwd_noalloc_max_bytes": (_SZ, []),
    "qlora_linear_fwd_noalloc": (ctypes.c_int, [_P, _I64, _P, _P, _P, ctypes.c_int, ctypes.c_float, _P, _P, _P]),
    "qlora_linear_set_workspace_bytes": (_SZ, [_I64, ctypes.c_int, _P, _I64, ctypes.c_int]),
    "qlora_linear_set_fwd": (ctypes.c_int, [_P, _I64, ctypes.c_int, _P, _P, _P, ctypes.c_int, ctypes.c_float, _P, _P,
                                            _P, _SZ, _P]),
    "qlora_linear_set_bwd": (ctypes.c_int, [_P, _P, _I64, ctypes.c_int, _P, _P, _P, ctypes.c_int, ctypes.c_float,
                                            _P, _P, _P, _P, _P, _SZ, _P]),
    "qlora_linear_dropout_workspace_bytes": (_SZ, [_I64, _I64, _I64, ctypes.c_int]),
    "qlora_linear_fwd_dropout": (ctypes.c_int, [_P, _I64, _P, _P, _P, ctypes.c_int, ctypes.c_float, ctypes.c_double,
                                                ctypes.c_uint64, _P, _P, _P, _SZ, _P]),
    "qlora_linear_bwd_dropout": (ctypes.c_int, [_P, _P, _I64, _P, _P, _P, ctypes.c_int, ctypes.c_float,
                                                ctypes.c_double, ctypes.c_uint64, _P, _P, _P, _P, _P, _SZ, _P]),
    "qlora_dropout_mask": (ctypes.c_int, [_P, _I64, _I64, ctypes.c_double, ctypes.c_uint64, _P, _P, _P]),
    "qlora_adamw_step": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _I64, ctypes.c_double, ctypes.c_double,
                                        ctypes.c_double, ctypes.c_double, ctypes.c_double, _P]),
    "qlora_act8_write": (ctypes.c_int, [_P, _P, _P]),
    "qlora_act8_read": (ctypes.c_int, [_P, _P, _P]),
    "qlora_linear_bwd_act8": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_float, _P, _P, _P, _P, _P, _SZ,
                                             _P]),
    "qlora_linear_set_bwd_act8": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, _P, _P, ctypes.c_int, ctypes.c_float, _P, _P,
                                                 _P, _P, _P, _SZ, _P]),
    "qlora_linear_set_act8_workspace_bytes": (_SZ, [_I64, ctypes.c_int, _P, _I64, ctypes.c_int]),
    "qlora_linear_set_act8_workspace_bound": (_SZ, [_I64, ctypes.c_int, ctypes.c_int]),
    "qlora_head_loss": (ctypes.c_int, [_P, _I64, _P, _I64, _I64, _P, _P, ctypes.c_float, _P, _P, _P, _P, _SZ, _P]),
    "qlora_head_loss_nf4": (ctypes.c_int, [_P, _I64, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P, _SZ, _P]),
    "qlora_head_loss_workspace_bytes": (_SZ, [_I64, _I64, _I64, ctypes.c_int, ctypes.c_int]),
    "qlora_rms_norm_fwd": (ctypes.c_int, [_P, _P, _I64, _I64, _P, ctypes.c_int, ctypes.c_float, _P, _P, _P, _P]),
    "qlora_rms_norm_bwd_workspace_bytes": (_SZ, [_I64, _I64]),
    "qlora_rms_norm_bwd": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _P, ctypes.c_int, ctypes.c_float, _P, _P, _P, _SZ,
                                          _P]),
    "qlora_gated_act_fwd": (ctypes.c_int, [_P, _P, _I64, _I64, ctypes.c_int, _P, _P, _P]),
    "qlora_gated_act_bwd": (ctypes.c_int, [_P, _P, _P, _I64, _I64, ctypes.c_int, _P, _P, _P]),
    "qlora_linear_gated_workspace_bytes": (_SZ, [_I64, _I64, _I64, ctypes.c_int]),
    "qlora_linear_gated_fwd": (ctypes.c_int, [_P, _I64, _P, _P, _P, ctypes.c_int, ctypes.c_float, ctypes.c_int, _P, _P,
                                              _P, _P, _P, _P, _SZ, _P]),
    "qlora_status_read": (ctypes.c_int, [_P, _P]),
    "qlora_kernel_timing_enable": (None, [ctypes.c_int]),
    "qlora_kernel_timing_read": (ctypes.c_int, [_P, _P]),
}


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_quantized_finetuning_quant_amd.build`")
        try:
            _torch()  # first: loaded before it, the library would bring in a HIP runtime beside torch's own
        except ImportError:
            pass
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise QloraError(status, where)


# ---------------------------------------------------------------- host helpers
def status_string(status: int) -> str:
    return lib().qlora_status_string(int(status)).decode()


def version() -> str:
    return lib().qlora_version().decode()


def nf4_sizes(n_out: int, n_in: int):
    cb, nb, ng = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().qlora_nf4_sizes(n_out, n_in, ctypes.byref(cb), ctypes.byref(nb), ctypes.byref(ng)), "nf4_sizes")
    return cb.value, nb.value, ng.value


def nf4_bytes(n_out: int, n_in: int, double_quant: bool = True) -> int:
    if double_quant:
        return int(lib().qlora_nf4_bytes(n_out, n_in))
    return int(lib().qlora_nf4_bytes_flags(n_out, n_in, QLORA_NF4_FP32_CONSTANTS))


def quantize_workspace_bytes(n_out: int, n_in: int) -> int:
    return int(lib().qlora_quantize_workspace_bytes(n_out, n_in))


def linear_workspace_bytes(tokens: int, n_out: int, n_in: int, r: int) -> int:
    return int(lib().qlora_linear_workspace_bytes(tokens, n_out, n_in, r))


TIMED_KINDS = ("qgemm_fwd", "qgemm_dx", "gemv_fwd", "gemv_bwd", "adamw")


def kernel_timing_enable(on: bool) -> None:
    """Bracket every main-kernel launch with HIP events on its stream (diagnostics)."""
    lib().qlora_kernel_timing_enable(1 if on else 0)


def kernel_timing_read():
    """-> {kind: (launches, total ms)} for the launches timed so far (then cleared)."""
    n = (ctypes.c_int64 * len(TIMED_KINDS))()
    ms = (ctypes.c_double * len(TIMED_KINDS))()
    _check(lib().qlora_kernel_timing_read(n, ms), "kernel_timing_read")
    return {k: (n[i], ms[i]) for i, k in enumerate(TIMED_KINDS)}


def nf4_codebook():
    buf = (ctypes.c_float * 16)()
    lib().qlora_nf4_codebook(buf)
    return list(buf)


# ------------------------------------------------------------- device helpers
_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch

        _TORCH = torch
    return _TORCH


def _stream(stream=None) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    c = _torch()._C
    # the current stream's handle without a Stream object around it (3 us of every call)
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _stream_on(dev, stream=None) -> int:
    """The stream's handle for a call on tensors of `dev`, which must be the current device (a launch goes
    to the current one, whatever device the pointers belong to)."""
    c = _torch()._C
    current = c._cuda_getDevice()
    if dev.index != current:
        raise ValueError(f"the tensors are on {dev}, the current device is cuda:{current}: call it under "
                         f"torch.cuda.device({dev.index})")
    if stream is None:
        return c._cuda_getCurrentRawStream(current)
    if stream.device != dev:
        raise ValueError(f"the tensors are on {dev}, the stream on {stream.device}")
    return int(stream.cuda_stream)


def _alloc_on(stream):
    """The context in which a call allocates what its caller did not give: the memory then belongs to the stream
    that the call runs on, where it may be given back as soon as the call returns."""
    return nullcontext() if stream is None else _torch().cuda.stream(stream)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


# The C ABI takes plain pointers and cannot check the extent of a buffer, so every tensor is
# checked here before a call: dtype, contiguity, exact shape, and the device of the packed
# weight.  A wrong tensor raises ValueError and nothing is launched.
_DT = {}  # dtype sets of the checks, filled on first use (torch is imported lazily)


def _dtypes():
    if not _DT:
        torch = _torch()
        _DT.update(tensor=torch.Tensor, bf16=(torch.bfloat16, torch.int16), f32=(torch.float32,),
                   i64=(torch.int64,), i8=(torch.int8,))
    return _DT


_TRUST = threading.local()


class trusted_calls:
    """Context manager: inside it the calls of this thread skip the per-tensor checks below (about
    1 us of host time per tensor, which is most of a few-token step's launch cost).  For loops that
    repeat calls on tensors already checked once (the same shapes, dtypes and device)."""

    def __enter__(self):
        self.prev = getattr(_TRUST, "on", False)
        _TRUST.on = True
        return self

    def __exit__(self, *exc):
        _TRUST.on = self.prev
        return False


class _NoChecks:
    __slots__ = ()

    def bf16(self, t, name, shape):
        pass

    def f32(self, t, name, shape):
        pass

    def i64(self, t, name, shape):
        pass

    def i8(self, t, name, shape):
        pass

    def done(self):
        pass


_NO_CHECKS = _NoChecks()


class _Args:
    """Checks of one call's tensors: dtype, exact shape and contiguity as each is named, then
    (done) that every one of them is on the packed weight's CUDA device."""

    __slots__ = ("device", "named")

    def __new__(cls, device):
        if getattr(_TRUST, "on", False):
            return _NO_CHECKS
        return super().__new__(cls)

    def __init__(self, device):
        self.device = device
        self.named = []

    def _check(self, t, name: str, shape, kind: str) -> None:
        dt = _DT or _dtypes()
        if isinstance(t, dt["tensor"]) and t.dtype in dt[kind] and t.shape == shape and t.is_contiguous():
            self.named.append((name, t))
            return
        if not isinstance(t, dt["tensor"]):
            raise ValueError(f"{name} must be a tensor")
        if t.dtype not in dt[kind]:
            raise ValueError(f"{name} must be {' or '.join(str(d) for d in dt[kind])}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")

    def bf16(self, t, name: str, shape) -> None:
        self._check(t, name, shape, "bf16")

    def f32(self, t, name: str, shape) -> None:
        self._check(t, name, shape, "f32")

    def i64(self, t, name: str, shape) -> None:
        self._check(t, name, shape, "i64")

    def i8(self, t, name: str, shape) -> None:
        self._check(t, name, shape, "i8")

    def done(self) -> None:
        dev = self.device
        cuda = dev.type == "cuda"
        for name, t in self.named:
            if not cuda or t.device != dev:
                raise ValueError(f"{name} must be on {dev}, not {t.device}")


def _workspace(ws, device, need) -> int:
    """Checks a caller's workspace (a contiguous uint8 CUDA tensor of at least need() bytes)."""
    if getattr(_TRUST, "on", False):
        return ws.numel()
    torch = _torch()
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.dim() != 1 or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous 1-D uint8 tensor")
    if ws.device.type != "cuda" or ws.device != device:
        raise ValueError(f"workspace must be on {device}, not {ws.device}")
    need = need()
    if ws.numel() < need:
        raise ValueError(f"workspace holds {ws.numel()} bytes, the call needs {need}")
    return ws.numel()


def _weight_device(q) -> "object":
    """The device of a packed weight (every call's tensors must be on it)."""
    dev = q.codes.device
    if dev.type != "cuda":
        raise ValueError(f"the packed weight must be on a CUDA device, not {dev}")
    return dev


@dataclass
class NF4Weight:
    """Device buffers of a packed weight (allocated by torch, owned by this object).

    double_quant=False: absmax_scale holds the nblocks fp32 block constants and
    absmax_fp8 / absmax_mean are None (QLORA_NF4_FP32_CONSTANTS)."""
    n_out: int
    n_in: int
    codes: "object"
    absmax_fp8: "object"
    absmax_scale: "object"
    absmax_mean: "object"
    double_quant: bool = True

    @classmethod
    def empty(cls, n_out: int, n_in: int, device="cuda", double_quant: bool = True):
        torch = _torch()
        cb, nb, ng = nf4_sizes(n_out, n_in)
        codes = torch.empty(cb, dtype=torch.uint8, device=device)
        if not double_quant:
            return cls(n_out, n_in, codes, None, torch.empty(nb, dtype=torch.float32, device=device), None, False)
        return cls(n_out, n_in, codes, torch.empty(nb, dtype=torch.uint8, device=device),
                   torch.empty(ng, dtype=torch.float32, device=device),
                   torch.empty(1, dtype=torch.float32, device=device))

    def struct(self) -> NF4WeightStruct:
        return NF4WeightStruct(self.n_out, self.n_in, _ptr(self.codes), _ptr(self.absmax_fp8),
                               _ptr(self.absmax_scale), _ptr(self.absmax_mean),
                               0 if self.double_quant else QLORA_NF4_FP32_CONSTANTS)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.codes, self.absmax_fp8, self.absmax_scale, self.absmax_mean) if t is not None)


def _bits(t):
    """bf16 tensor -> the same memory viewed as int16 (no copy)."""
    torch = _torch()
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def quantize(w, out: NF4Weight = None, workspace=None, stream=None, double_quant: bool = True) -> NF4Weight:
    """Quantize a [n_out x n_in] fp32 or bf16 CUDA tensor to NF4 + FP8 double quantization
    (double_quant=False: NF4 + fp32 block constants; ignored when `out` is given, whose
    storage form decides)."""
    torch = _torch()
    if w.dim() != 2 or not w.is_contiguous():
        raise ValueError("w must be a contiguous 2-D tensor")
    dtype = {torch.float32: QLORA_F32, torch.bfloat16: QLORA_BF16}.get(w.dtype)
    if dtype is None:
        raise ValueError("w must be float32 or bfloat16")
    n_out, n_in = w.shape
    if w.device.type != "cuda":
        raise ValueError(f"w must be on a CUDA device, not {w.device}")
    q = out if out is not None else NF4Weight.empty(n_out, n_in, w.device, double_quant=double_quant)
    if (q.n_out, q.n_in) != (n_out, n_in) or _weight_device(q) != w.device:
        raise ValueError("out must be a packed weight of w's shape on w's device")
    wsb = quantize_workspace_bytes(n_out, n_in)
    ws = workspace if workspace is not None else torch.empty(wsb, dtype=torch.uint8, device=w.device)
    wsn = _workspace(ws, w.device, lambda: wsb)
    st = q.struct()
    _check(lib().qlora_quantize(_ptr(w), dtype, ctypes.byref(st), _ptr(ws), wsn, _stream(stream)), "qlora_quantize")
    q.last_workspace = ws
    return q


def status_read(workspace, stream=None) -> int:
    """Synchronise and return the status word a call left in `workspace` (0 = ok)."""
    return int(lib().qlora_status_read(_ptr(workspace), _stream(stream)))


def dequantize(q: NF4Weight, out=None, stream=None):
    torch = _torch()
    dev = _weight_device(q)
    y = out if out is not None else torch.empty((q.n_out, q.n_in), dtype=torch.bfloat16, device=dev)
    chk = _Args(dev)
    chk.bf16(y, "out", (q.n_out, q.n_in))
    chk.done()
    st = q.struct()
    _check(lib().qlora_dequantize(ctypes.byref(st), _ptr(y), _stream(stream)), "qlora_dequantize")
    return y


def dequantize_many(qs, outs=None, stream=None):
    """Decode several packed weights (up to 8) in one launch; returns the bf16 tensors."""
    torch = _torch()
    outs = outs if outs is not None else [torch.empty((q.n_out, q.n_in), dtype=torch.bfloat16, device=q.codes.device)
                                          for q in qs]
    _check_list(outs, len(qs), "outs")
    for i, (q, o) in enumerate(zip(qs, outs)):
        chk = _Args(_weight_device(q))
        chk.bf16(o, f"outs[{i}]", (q.n_out, q.n_in))
        chk.done()
    st = (NF4WeightStruct * len(qs))(*[q.struct() for q in qs])
    ptrs = (ctypes.c_void_p * len(outs))(*[_ptr(o) for o in outs])
    _check(lib().qlora_dequantize_many(st, len(qs), ptrs, _stream(stream)), "qlora_dequantize_many")
    return outs


def linear_workspace(tokens: int, n_out: int, n_in: int, r: int, device="cuda"):
    """A workspace for the linear calls (reusable by successive calls on one stream)."""
    torch = _torch()
    return torch.empty(max(linear_workspace_bytes(tokens, n_out, n_in, r), 1), dtype=torch.uint8, device=device)


def linear_fwd(x, q: NF4Weight, A, B, scale: float, y=None, u_out=None, save_u=True, workspace=None,
               stream=None):
    """y = x W_hat^T + scale (x A^T) B^T (bf16); returns (y, u or None)."""
    torch = _torch()
    T, r = _linear_dims(x, A, q)
    dev = _weight_device(q)
    chk = _Args(dev)
    chk.bf16(x, "x", (T, q.n_in))
    chk.bf16(A, "A", (r, q.n_in))
    chk.bf16(B, "B", (q.n_out, r))
    y = y if y is not None else torch.empty((T, q.n_out), dtype=torch.bfloat16, device=dev)
    chk.bf16(y, "y", (T, q.n_out))
    if save_u and u_out is None:
        u_out = torch.empty((T, r), dtype=torch.bfloat16, device=dev)
    if u_out is not None:
        chk.bf16(u_out, "u_out", (T, r))
    chk.done()
    ws = workspace if workspace is not None else linear_workspace(T, q.n_out, q.n_in, r, dev)
    wsb = _workspace(ws, dev, lambda: linear_workspace_bytes(T, q.n_out, q.n_in, r))
    st = q.struct()
    _check(lib().qlora_linear_fwd(_ptr(x), T, ctypes.byref(st), _ptr(A), _ptr(B), r, float(scale), _ptr(y),
                                  _ptr(u_out), _ptr(ws), wsb, _stream(stream)), "qlora_linear_fwd")
    return y, u_out


def linear_fwd_noalloc(x, q: NF4Weight, A, B, scale: float, y, u_out=None, stream=None):
    """linear_fwd on the library's fixed per-GPU scratch array instead of a workspace (for callers
    that cannot allocate): y (and u_out, if given) are the caller's; nothing is allocated here.
    Calls that may overlap in time on one GPU share the array and must be ordered."""
    T, r = _linear_dims(x, A, q)
    dev = _weight_device(q)
    chk = _Args(dev)
    chk.bf16(x, "x", (T, q.n_in))
    chk.bf16(A, "A", (r, q.n_in))
    chk.bf16(B, "B", (q.n_out, r))
    chk.bf16(y, "y", (T, q.n_out))
    if u_out is not None:
        chk.bf16(u_out, "u_out", (T, r))
    chk.done()
    st = q.struct()
    _check(lib().qlora_linear_fwd_noalloc(_ptr(x), T, ctypes.byref(st), _ptr(A), _ptr(B), r, float(scale), _ptr(y),
                                          _ptr(u_out), _stream(stream)), "qlora_linear_fwd_noalloc")
    return y, u_out


def linear_fwd_noalloc_max_bytes() -> int:
    return int(lib().qlora_linear_fwd_noalloc_max_bytes())


def _linear_dims(x, A, q):
    """(T, r) of a linear call from x [T x n_in] and A [r x n_in]."""
    if x.dim() != 2 or A.dim() != 2:
        raise ValueError("x and A must be 2-D")
    return int(x.shape[0]), int(A.shape[0])


def _check_bwd(dy, x, q, A, B, u, chk):
    T, r = _linear_dims(x, A, q)
    chk.bf16(dy, "dy", (T, q.n_out))
    chk.bf16(x, "x", (T, q.n_in))
    chk.bf16(A, "A", (r, q.n_in))
    chk.bf16(B, "B", (q.n_out, r))
    if u is not None:
        chk.bf16(u, "u", (T, r))
    return T, r


def _check_grads(grad_x, grad_A, grad_B, T, r, q, chk):
    if grad_x is not None:
        chk.bf16(grad_x, "grad_x", (T, q.n_in))
    chk.f32(grad_A, "grad_A", (r, q.n_in))
    chk.f32(grad_B, "grad_B", (q.n_out, r))
    chk.done()


def linear_bwd(dy, x, q: NF4Weight, A, B, scale: float, u=None, need_grad_x=True, grad_x=None, grad_A=None,
               grad_B=None, workspace=None, stream=None):
    """Returns (grad_x bf16 or None, grad_A fp32, grad_B fp32)."""
    torch = _torch()
    dev = _weight_device(q)
    chk = _Args(dev)
    T, r = _check_bwd(dy, x, q, A, B, u, chk)
    if need_grad_x and grad_x is None:
        grad_x = torch.empty((T, q.n_in), dtype=torch.bfloat16, device=dev)
    if not need_grad_x:
        grad_x = None
    grad_A = grad_A if grad_A is not None else torch.empty((r, q.n_in), dtype=torch.float32, device=dev)
    grad_B = grad_B if grad_B is not None else torch.empty((q.n_out, r), dtype=torch.float32, device=dev)
    _check_grads(grad_x, grad_A, grad_B, T, r, q, chk)
    ws = workspace if workspace is not None else linear_workspace(T, q.n_out, q.n_in, r, dev)
    wsb = _workspace(ws, dev, lambda: linear_workspace_bytes(T, q.n_out, q.n_in, r))
    st = q.struct()
    _check(lib().qlora_linear_bwd(_ptr(dy), _ptr(x), T, ctypes.byref(st), _ptr(A), _ptr(B), r, float(scale),
                                  _ptr(u), _ptr(grad_x), _ptr(grad_A), _ptr(grad_B), _ptr(ws), wsb,
                                  _stream(stream)), "qlora_linear_bwd")
    return grad_x, grad_A, grad_B


def adamw_step(param, param_bf16, grad, exp_avg, exp_avg_sq, step: int, lr: float, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0, stream=None) -> None:
    """One AdamW update of a flat fp32 adapter buffer, in place (see qlora_adamw_step).

    param, grad, exp_avg, exp_avg_sq: contiguous float32 tensors of n elements;
    param_bf16: bfloat16 (or int16) tensor of n elements.  The states may be
    pinned host tensors (``pin_memory=True``): the kernel reads them in place.
    """
    torch = _torch()
    n = param.numel()
    for name, t, dt in (("param", param, torch.float32), ("grad", grad, torch.float32),
                        ("exp_avg", exp_avg, torch.float32), ("exp_avg_sq", exp_avg_sq, torch.float32)):
        if t.dtype != dt or not t.is_contiguous() or t.numel() != n:
            raise ValueError(f"{name} must be a contiguous float32 tensor of {n} elements")
    if param_bf16.dtype not in (torch.bfloat16, torch.int16) or not param_bf16.is_contiguous() \
            or param_bf16.numel() != n:
        raise ValueError(f"param_bf16 must be a contiguous bfloat16 tensor of {n} elements")
    _check(lib().qlora_adamw_step(_ptr(param), _ptr(param_bf16), _ptr(grad), _ptr(exp_avg), _ptr(exp_avg_sq), n,
                                  int(step), float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                                  _stream(stream)), "qlora_adamw_step")


# ------------------------------------------------------------------ LoRA dropout
def linear_dropout_workspace_bytes(tokens: int, n_out: int, n_in: int, r: int) -> int:
    return int(lib().qlora_linear_dropout_workspace_bytes(tokens, n_out, n_in, r))


def linear_dropout_workspace(tokens: int, n_out: int, n_in: int, r: int, device="cuda"):
    torch = _torch()
    return torch.empty(max(linear_dropout_workspace_bytes(tokens, n_out, n_in, r), 1), dtype=torch.uint8,
                       device=device)


def linear_fwd_dropout(x, q: NF4Weight, A, B, scale: float, p: float, seed: int, y=None, u_out=None, save_u=True,
                       workspace=None, stream=None):
    """linear_fwd with LoRA dropout of probability p on the adapter input (mask from seed)."""
    torch = _torch()
    T, r = _linear_dims(x, A, q)
    dev = _weight_device(q)
    chk = _Args(dev)
    chk.bf16(x, "x", (T, q.n_in))
    chk.bf16(A, "A", (r, q.n_in))
    chk.bf16(B, "B", (q.n_out, r))
    y = y if y is not None else torch.empty((T, q.n_out), dtype=torch.bfloat16, device=dev)
    chk.bf16(y, "y", (T, q.n_out))
    if save_u and u_out is None:
        u_out = torch.empty((T, r), dtype=torch.bfloat16, device=dev)
    if u_out is not None:
        chk.bf16(u_out, "u_out", (T, r))
    chk.done()
    ws = workspace if workspace is not None else linear_dropout_workspace(T, q.n_out, q.n_in, r, dev)
    wsb = _workspace(ws, dev, lambda: linear_dropout_workspace_bytes(T, q.n_out, q.n_in, r))
    st = q.struct()
    _check(lib().qlora_linear_fwd_dropout(_ptr(x), T, ctypes.byref(st), _ptr(A), _ptr(B), r, float(scale), float(p),
                                          int(seed), _ptr(y), _ptr(u_out), _ptr(ws), wsb, _stream(stream)),
           "qlora_linear_fwd_dropout")
    return y, u_out


def linear_bwd_dropout(dy, x, q: NF4Weight, A, B, scale: float, p: float, seed: int, u=None, need_grad_x=True,
                       grad_x=None, grad_A=None, grad_B=None, workspace=None, stream=None):
    """linear_bwd with the forward's dropout mask (same p and seed)."""
    torch = _torch()
    dev = _weight_device(q)
    chk = _Args(dev)
    T, r = _check_bwd(dy, x, q, A, B, u, chk)
    if need_grad_x and grad_x is None:
        grad_x = torch.empty((T, q.n_in), dtype=torch.bfloat16, device=dev)
    if not need_grad_x:
        grad_x = None
    grad_A = grad_A if grad_A is not None else torch.empty((r, q.n_in), dtype=torch.float32, device=dev)
    grad_B = grad_B if grad_B is not None else torch.empty((q.n_out, r), dtype=torch.float32, device=dev)
    _check_grads(grad_x, grad_A, grad_B, T, r, q, chk)
    ws = workspace if workspace is not None else linear_dropout_workspace(T, q.n_out, q.n_in, r, dev)
    wsb = _workspace(ws, dev, lambda: linear_dropout_workspace_bytes(T, q.n_out, q.n_in, r))
    st = q.struct()
    _check(lib().qlora_linear_bwd_dropout(_ptr(dy), _ptr(x), T, ctypes.byref(st), _ptr(A), _ptr(B), r, float(scale),
                                          float(p), int(seed), _ptr(u), _ptr(grad_x), _ptr(grad_A), _ptr(grad_B),
                                          _ptr(ws), wsb, _stream(stream)), "qlora_linear_bwd_dropout")
    return grad_x, grad_A, grad_B


def dropout_mask(x, p: float, seed: int, stream=None):
    """(keep_words [ceil(T/32) x K] int32, x_drop [T x K] bf16) for a [T x K] bf16 tensor."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    T, K = x.shape
    chk = _Args(x.device)
    chk.bf16(x, "x", (T, K))
    chk.done()
    keep = torch.empty(((T + 31) // 32, K), dtype=torch.int32, device=x.device)
    xd = torch.empty((T, K), dtype=torch.bfloat16, device=x.device)
    _check(lib().qlora_dropout_mask(_ptr(x), T, K, float(p), int(seed), _ptr(keep), _ptr(xd), _stream(stream)),
           "qlora_dropout_mask")
    return keep, xd


# ------------------------------------------------------------ projection sets
def _ptrs(ts):
    return (ctypes.c_void_p * len(ts))(*[_ptr(t) for t in ts])


def linear_set_workspace_bytes(tokens: int, n_outs, n_in: int, r: int) -> int:
    arr = (ctypes.c_int64 * len(n_outs))(*n_outs)
    return int(lib().qlora_linear_set_workspace_bytes(tokens, len(n_outs), arr, n_in, r))


def linear_set_workspace(tokens: int, n_outs, n_in: int, r: int, device="cuda"):
    torch = _torch()
    return torch.empty(max(linear_set_workspace_bytes(tokens, n_outs, n_in, r), 1), dtype=torch.uint8, device=device)


def linear_set_fwd(x, qs, A_set, Bs, scale: float, ys=None, u_out=None, save_u=True, workspace=None, stream=None):
    """Projection set forward: y_i = x W_hat_i^T + scale (x A_i^T) B_i^T for every member, with
    A_set [count r x n_in] the members' A matrices back to back.  Returns (ys, u_set or None)."""
    torch = _torch()
    T, count, r, dev, chk = _set_dims(x, qs, A_set)
    _check_list(Bs, count, "Bs")
    for i, (q, b) in enumerate(zip(qs, Bs)):
        chk.bf16(b, f"Bs[{i}]", (q.n_out, r))
    ys = ys if ys is not None else [torch.empty((T, q.n_out), dtype=torch.bfloat16, device=dev) for q in qs]
    _check_list(ys, count, "ys")
    for i, (q, y) in enumerate(zip(qs, ys)):
        chk.bf16(y, f"ys[{i}]", (T, q.n_out))
    if save_u and u_out is None:
        u_out = torch.empty((T, count * r), dtype=torch.bfloat16, device=dev)
    if u_out is not None:
        chk.bf16(u_out, "u_out", (T, count * r))
    chk.done()
    n_outs = [q.n_out for q in qs]
    ws = workspace if workspace is not None else linear_set_workspace(T, n_outs, qs[0].n_in, r, dev)
    wsb = _workspace(ws, dev, lambda: linear_set_workspace_bytes(T, n_outs, qs[0].n_in, r))
    st = (NF4WeightStruct * count)(*[q.struct() for q in qs])
    _check(lib().qlora_linear_set_fwd(_ptr(x), T, count, st, _ptr(A_set), _ptrs(Bs), r, float(scale), _ptrs(ys),
                                      _ptr(u_out), _ptr(ws), wsb, _stream(stream)), "qlora_linear_set_fwd")
    return ys, u_out


def _check_list(ts, count: int, name: str) -> None:
    if len(ts) != count:
        raise ValueError(f"{name} must hold {count} tensors, not {len(ts)}")


def _set_dims(x, qs, A_set, act8=None):
    """(T, count, r, device, checker) of a projection-set call; A_set must hold count whole [r x n_in] blocks.
    act8: the checkpoint that x is the codes of."""
    count = len(qs)
    if count < 1:
        raise ValueError("a projection set needs at least one member")
    dev = _weight_device(qs[0])
    for i, q in enumerate(qs):
        if q.n_in != qs[0].n_in:
            raise ValueError(f"member {i} has n_in {q.n_in}, member 0 has {qs[0].n_in}")
        if _weight_device(q) != dev:
            raise ValueError(f"member {i} is on {q.codes.device}, member 0 on {dev}")
    if x.dim() != 2 or A_set.dim() != 2:
        raise ValueError("x and A_set must be 2-D")
    if A_set.shape[0] % count:
        raise ValueError(f"A_set has {A_set.shape[0]} rows, not a multiple of the {count} members")
    T, r = int(x.shape[0]), int(A_set.shape[0]) // count
    chk = _Args(dev)
    if act8 is None:
        chk.bf16(x, "x", (T, qs[0].n_in))
    elif _check_act8(act8, chk)[1] != qs[0].n_in:
        raise ValueError(f"codes must have {qs[0].n_in} columns, not {x.shape[1]}")
    chk.bf16(A_set, "A_set", (count * r, qs[0].n_in))
    return T, count, r, dev, chk


def linear_set_bwd(dys, x, qs, A_set, Bs, scale: float, u=None, need_grad_x=True, grad_x=None, grad_A_set=None,
                   grad_Bs=None, workspace=None, stream=None):
    """Projection set backward: (grad_x summed over the members or None, grad_A_set, [grad_B_i])."""
    torch = _torch()
    T, count, r, dev, chk = _set_dims(x, qs, A_set)
    _check_list(dys, count, "dys")
    _check_list(Bs, count, "Bs")
    for i, (q, d, b) in enumerate(zip(qs, dys, Bs)):
        chk.bf16(d, f"dys[{i}]", (T, q.n_out))
        chk.bf16(b, f"Bs[{i}]", (q.n_out, r))
    if u is not None:
        chk.bf16(u, "u", (T, count * r))
    if need_grad_x and grad_x is None:
        grad_x = torch.empty((T, qs[0].n_in), dtype=torch.bfloat16, device=dev)
    if not need_grad_x:
        grad_x = None
    if grad_x is not None:
        chk.bf16(grad_x, "grad_x", (T, qs[0].n_in))
    grad_A_set = grad_A_set if grad_A_set is not None else torch.empty((count * r, qs[0].n_in), dtype=torch.float32,
                                                                       device=dev)
    chk.f32(grad_A_set, "grad_A_set", (count * r, qs[0].n_in))
    grad_Bs = grad_Bs if grad_Bs is not None else [torch.empty((q.n_out, r), dtype=torch.float32, device=dev)
                                                   for q in qs]
    _check_list(grad_Bs, count, "grad_Bs")
    for i, (q, g) in enumerate(zip(qs, grad_Bs)):
        chk.f32(g, f"grad_Bs[{i}]", (q.n_out, r))
    chk.done()
    n_outs = [q.n_out for q in qs]
    ws = workspace if workspace is not None else linear_set_workspace(T, n_outs, qs[0].n_in, r, dev)
    wsb = _workspace(ws, dev, lambda: linear_set_workspace_bytes(T, n_outs, qs[0].n_in, r))
    st = (NF4WeightStruct * count)(*[q.struct() for q in qs])
    _check(lib().qlora_linear_set_bwd(_ptrs(dys), _ptr(x), T, count, st, _ptr(A_set), _ptrs(Bs), r, float(scale),
                                      _ptr(u), _ptr(grad_x), _ptr(grad_A_set), _ptrs(grad_Bs), _ptr(ws), wsb,
                                      _stream(stream)), "qlora_linear_set_bwd")
    return grad_x, grad_A_set, grad_Bs


# -------------------------------------------------- 8-bit activation checkpoints
@dataclass
class Act8:
    """An activation [T x K] in 8.5 bits per value: codes int8 [T x K], scale fp32 [T x K / 64]."""
    codes: "object"
    scale: "object"

    @classmethod
    def empty(cls, tokens: int, dim: int, device="cuda"):
        torch = _torch()
        if dim % 64:
            raise ValueError(f"dim must be a multiple of 64, not {dim}")
        return cls(torch.empty((tokens, dim), dtype=torch.int8, device=device),
                   torch.empty((tokens, dim // 64), dtype=torch.float32, device=device))

    def struct(self) -> Act8Struct:
        return Act8Struct(*self.codes.shape, self.codes.data_ptr(), self.scale.data_ptr())

    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scale.numel()


def _check_act8(a: Act8, chk):
    """(T, K) of a checkpoint whose tensors fit each other."""
    if a.codes.dim() != 2:
        raise ValueError("codes must be 2-D")
    T, K = a.codes.shape
    if K % 64:
        raise ValueError(f"codes must have a multiple of 64 columns, not {K}")
    chk.i8(a.codes, "codes", (T, K))
    chk.f32(a.scale, "scale", (T, K // 64))
    return T, K


def act8_write(x, out: Act8 = None, stream=None) -> Act8:
    """Keep a [T x K] bf16 activation (K % 64 == 0) as an 8-bit checkpoint: per 64 columns one fp32 scale,
    absmax / 127, and the nearest codes."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    T, K = x.shape
    chk = _Args(x.device)
    chk.bf16(x, "x", (T, K))
    if out is not None and _check_act8(out, chk) != (T, K):
        raise ValueError(f"out must hold {T} x {K} values, not {out.codes.shape[0]} x {out.codes.shape[1]}")
    chk.done()
    handle = _stream_on(x.device, stream)
    a = out
    if a is None:
        with _alloc_on(stream):
            a = Act8.empty(T, K, x.device)
    st = a.struct()
    _check(lib().qlora_act8_write(x.data_ptr(), ctypes.byref(st), handle), "qlora_act8_write")
    return a


def act8_read(a: Act8, out=None, stream=None):
    """The bf16 values a checkpoint stands for."""
    torch = _torch()
    chk = _Args(a.codes.device)
    T, K = _check_act8(a, chk)
    if out is not None:
        chk.bf16(out, "out", (T, K))
    chk.done()
    handle = _stream_on(a.codes.device, stream)
    y = out
    if y is None:
        with _alloc_on(stream):
            y = torch.empty((T, K), dtype=torch.bfloat16, device=a.codes.device)
    st = a.struct()
    _check(lib().qlora_act8_read(ctypes.byref(st), y.data_ptr(), handle), "qlora_act8_read")
    return y


@functools.lru_cache(maxsize=1024)
def _act8_bytes(tokens: int, n_outs: tuple, n_in: int, r: int) -> int:
    arr = (ctypes.c_int64 * len(n_outs))(*n_outs)
    return int(lib().qlora_linear_set_act8_workspace_bytes(tokens, len(n_outs), arr, n_in, r))


def linear_set_act8_workspace_bytes(tokens: int, n_outs, n_in: int, r: int) -> int:
    return _act8_bytes(tokens, tuple(n_outs), n_in, r)


@functools.lru_cache(maxsize=1024)
def linear_set_act8_workspace_bound(tokens: int, members: int, r: int) -> int:
    """Bytes of a workspace that serves every linear_set_bwd_act8 (members = 1: linear_bwd_act8) of up to `tokens`
    tokens, whatever the weights' sizes; where it is less than linear_set_act8_workspace_bytes, grad_x may take longer."""
    return int(lib().qlora_linear_set_act8_workspace_bound(tokens, members, r))


def linear_set_act8_workspace(tokens: int, n_outs, n_in: int, r: int, device="cuda"):
    """A workspace for linear_set_bwd_act8, and with one n_out for linear_bwd_act8, of exactly these sizes (fewer
    tokens may need more; linear_set_act8_workspace_bound has the bytes that serve them all)."""
    torch = _torch()
    return torch.empty(max(linear_set_act8_workspace_bytes(tokens, n_outs, n_in, r), 1), dtype=torch.uint8,
                       device=device)


def linear_bwd_act8(dy, a: Act8, q: NF4Weight, A, B, scale: float, u, need_grad_x=True, grad_x=None, grad_A=None,
                    grad_B=None, workspace=None, stream=None):
    """linear_bwd with the checkpoint `a` of the layer's input in place of x; u is the forward's.
    Returns (grad_x bf16 or None, grad_A fp32, grad_B fp32)."""
    grad_x, grad_A, grad_Bs = linear_set_bwd_act8([dy], a, [q], A, [B], scale, u, need_grad_x, grad_x, grad_A,
                                                  [grad_B] if grad_B is not None else None, workspace, stream)
    return grad_x, grad_A, grad_Bs[0]


def linear_set_bwd_act8(dys, a: Act8, qs, A_set, Bs, scale: float, u, need_grad_x=True, grad_x=None, grad_A_set=None,
                        grad_Bs=None, workspace=None, stream=None):
    """linear_set_bwd with the checkpoint `a` of the shared input in place of x; u is the forward's.
    Returns (grad_x summed over the members or None, grad_A_set, [grad_B_i])."""
    torch = _torch()
    T, count, r, dev, chk = _set_dims(a.codes, qs, A_set, act8=a)
    _check_list(dys, count, "dys")
    _check_list(Bs, count, "Bs")
    for i, (q, d, b) in enumerate(zip(qs, dys, Bs)):
        chk.bf16(d, f"dys[{i}]", (T, q.n_out))
        chk.bf16(b, f"Bs[{i}]", (q.n_out, r))
    chk.bf16(u, "u", (T, count * r))
    n_in = qs[0].n_in
    if not need_grad_x:
        grad_x = None
    elif grad_x is not None:
        chk.bf16(grad_x, "grad_x", (T, n_in))
    if grad_A_set is not None:
        chk.f32(grad_A_set, "grad_A_set", (count * r, n_in))
    if grad_Bs is not None:
        _check_list(grad_Bs, count, "grad_Bs")
        for i, (q, g) in enumerate(zip(qs, grad_Bs)):
            chk.f32(g, f"grad_Bs[{i}]", (q.n_out, r))
    chk.done()
    handle = _stream_on(dev, stream)
    n_outs = [q.n_out for q in qs]
    with _alloc_on(stream):
        if need_grad_x and grad_x is None:
            grad_x = torch.empty((T, n_in), dtype=torch.bfloat16, device=dev)
        if grad_A_set is None:
            grad_A_set = torch.empty((count * r, n_in), dtype=torch.float32, device=dev)
        if grad_Bs is None:
            grad_Bs = [torch.empty((q.n_out, r), dtype=torch.float32, device=dev) for q in qs]
        if workspace is None:
            wsb = linear_set_act8_workspace_bytes(T, n_outs, n_in, r)
            if not need_grad_x:  # what only grad_x needs is left out
                wsb = min(wsb, linear_set_act8_workspace_bound(T, count, r))
            ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
        else:
            ws = workspace
            wsb = _workspace(ws, dev, lambda: min(linear_set_act8_workspace_bytes(T, n_outs, n_in, r),
                                                  linear_set_act8_workspace_bound(T, count, r)))
    st = (NF4WeightStruct * count)(*[q.struct() for q in qs])
    sa = a.struct()
    _check(lib().qlora_linear_set_bwd_act8(_ptrs(dys), ctypes.byref(sa), count, st, _ptr(A_set), _ptrs(Bs), r,
                                           float(scale), _ptr(u), _ptr(grad_x), _ptr(grad_A_set), _ptrs(grad_Bs),
                                           _ptr(ws), wsb, handle), "qlora_linear_set_bwd_act8")
    return grad_x, grad_A_set, grad_Bs


# ----------------------------------------------------------- the loss of the head
@functools.lru_cache(maxsize=1024)
def head_loss_workspace_bytes(tokens: int, vocab: int, dim: int, grad: bool = True, packed: bool = False) -> int:
    return int(lib().qlora_head_loss_workspace_bytes(tokens, vocab, dim, int(grad), int(packed)))


def head_loss_workspace(tokens: int, vocab: int, dim: int, grad: bool = True, packed: bool = False, device="cuda"):
    """A workspace for head_loss of exactly these sizes (reusable by successive calls on one stream; fewer tokens
    may need more)."""
    torch = _torch()
    return torch.empty(max(head_loss_workspace_bytes(tokens, vocab, dim, grad, packed), 1), dtype=torch.uint8,
                       device=device)


def head_loss(h, head, target, scale: float = 1.0, weight=None, loss=None, lse=None, grad_h=None, need_grad=True,
              workspace=None, stream=None):
    """Softmax cross entropy of a frozen language-model head over its vocabulary, the logits never held;
    returns (loss, lse, grad_h or None).

    h [T x D] bf16; head: a bf16 tensor [V x D] or a packed NF4Weight; target [T] int64, negative where a
    token carries no loss.  loss and lse [T] fp32 are per token (target, weight, loss and lse may be views at any
    offset, which are copied; the matrices lie on 16-byte boundaries); grad_h [T x D] bf16 is the gradient of
    sum_t scale weight_t loss_t (weight [T] fp32, default ones).  A target >= V gives NaN, and
    status_read(workspace) then returns QLORA_ERR_VALUE (8)."""
    torch = _torch()
    packed = isinstance(head, NF4Weight)
    if h.dim() != 2 or not (packed or head.dim() == 2):
        raise ValueError("h and head must be 2-D")
    T, D = int(h.shape[0]), int(h.shape[1])
    V = head.n_out if packed else int(head.shape[0])
    dev = _weight_device(head) if packed else head.device
    chk = _Args(dev)
    chk.bf16(h, "h", (T, head.n_in if packed else D))
    if not packed:
        chk.bf16(head, "head", (V, D))
    chk.i64(target, "target", (T,))
    if weight is not None:
        chk.f32(weight, "weight", (T,))
    if loss is not None:
        chk.f32(loss, "loss", (T,))
    if lse is not None:
        chk.f32(lse, "lse", (T,))
    if not need_grad:
        grad_h = None
    elif grad_h is not None:
        chk.bf16(grad_h, "grad_h", (T, D))
    chk.done()
    handle = _stream_on(dev, stream)
    with _alloc_on(stream):
        if loss is None:
            loss = torch.empty(T, dtype=torch.float32, device=dev)
        if lse is None:
            lse = torch.empty(T, dtype=torch.float32, device=dev)
        if need_grad and grad_h is None:
            grad_h = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
        if workspace is None:
            ws = head_loss_workspace(T, V, D, need_grad, packed, dev)
            wsb = ws.numel()
        else:
            ws = workspace
            wsb = _workspace(ws, dev, lambda: head_loss_workspace_bytes(T, V, D, need_grad, packed))
        vectors = [target, weight, loss, lse]
        ptrs = [target.data_ptr(), _ptr(weight), loss.data_ptr(), lse.data_ptr()]
        if (ptrs[0] | ptrs[1] | ptrs[2] | ptrs[3]) & 15:
            # the C ABI takes 16-byte aligned pointers; labels[1:] and the like go through copies of T values
            for i in range(4):
                if ptrs[i] & 15:
                    vectors[i] = vectors[i].clone() if i < 2 else torch.empty_like(vectors[i])
                    ptrs[i] = vectors[i].data_ptr()
        if packed:
            st = head.struct()
            _check(lib().qlora_head_loss_nf4(_ptr(h), T, ctypes.byref(st), ptrs[0], ptrs[1], float(scale), ptrs[2], ptrs[3],
                                             _ptr(grad_h), _ptr(ws), wsb, handle), "qlora_head_loss_nf4")
        else:
            _check(lib().qlora_head_loss(_ptr(h), T, _ptr(head), V, D, ptrs[0], ptrs[1], float(scale), ptrs[2], ptrs[3],
                                         _ptr(grad_h), _ptr(ws), wsb, handle), "qlora_head_loss")
        if vectors[2] is not loss:
            loss.copy_(vectors[2])
        if vectors[3] is not lse:
            lse.copy_(vectors[3])
    return loss, lse, grad_h


# ------------------------------------- around the linears of a feed-forward block
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}


def _activation(name: str) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, not {name!r}")
    return code


def _rows(x, name: str):
    """(T, K) of an activation that a call may keep as an 8-bit checkpoint."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    T, K = x.shape
    if K % 64:
        raise ValueError(f"{name} must have a multiple of 64 columns, not {K}")
    return T, K


def _bf16_like(x):
    """A new bf16 tensor of x's shape, x checked already (empty_like takes two thirds of empty's time)."""
    torch = _torch()
    return torch.empty_like(x) if x.dtype is torch.bfloat16 else torch.empty_like(x, dtype=torch.bfloat16)


def _norm_weight(weight, chk, D: int) -> int:
    """The dtype code of a norm's weight [D]."""
    if weight.dtype == _torch().float32:
        chk.f32(weight, "weight", (D,))
        return QLORA_F32
    chk.bf16(weight, "weight", (D,))
    return QLORA_BF16


def _out8(act8, T: int, K: int, chk) -> None:
    if act8 is not None and _check_act8(act8, chk) != (T, K):
        raise ValueError(f"act8 must hold {T} x {K} values, not {act8.codes.shape[0]} x {act8.codes.shape[1]}")


def _ref8(act8):
    return None if act8 is None else ctypes.byref(act8.struct())


def rms_norm_fwd(x, weight, eps: float = 1e-6, residual=None, s=None, y=None, need_y=True, act8: Act8 = None,
                 need_act8=False, stream=None):
    """Root-mean-square norm of a [T x D] bf16 activation, D % 64 == 0: s = bf16(x + residual) (x itself without
    residual) and y = bf16(weight (s / sqrt(mean s^2 + eps))), with weight [D] bf16 or fp32.  Returns (y, s, act8):
    y is None with need_y=False, act8 the 8-bit checkpoint of y where it is given or need_act8.  s may be the
    residual or x, which the sum then replaces."""
    T, D = _rows(x, "x")
    dev = x.device
    chk = _Args(dev)
    chk.bf16(x, "x", (T, D))
    dtype = _norm_weight(weight, chk, D)
    if residual is not None:
        chk.bf16(residual, "residual", (T, D))
        if s is not None:
            chk.bf16(s, "s", (T, D))
    elif s is not None:
        raise ValueError("s is the sum with a residual: without one it is x")
    need_act8 = need_act8 or act8 is not None
    if not need_y:
        y = None
        if not need_act8:
            raise ValueError("need_y=False needs an 8-bit result")
    elif y is not None:
        chk.bf16(y, "y", (T, D))
    _out8(act8, T, D, chk)
    chk.done()
    handle = _stream_on(dev, stream)
    with _alloc_on(stream):
        if residual is not None and s is None:
            s = _bf16_like(x)
        if need_y and y is None:
            y = _bf16_like(x)
        if need_act8 and act8 is None:
            act8 = Act8.empty(T, D, dev)
    _check(lib().qlora_rms_norm_fwd(x.data_ptr(), _ptr(residual), T, D, weight.data_ptr(), dtype, float(eps), _ptr(s),
                                    _ptr(y), _ref8(act8), handle), "qlora_rms_norm_fwd")
    return y, x if s is None else s, act8


@functools.lru_cache(maxsize=1024)
def rms_norm_bwd_workspace_bytes(tokens: int, dim: int) -> int:
    return int(lib().qlora_rms_norm_bwd_workspace_bytes(tokens, dim))


def rms_norm_bwd_workspace(tokens: int, dim: int, device="cuda"):
    """A workspace for rms_norm_bwd with the weight's gradient (one without it needs none)."""
    torch = _torch()
    return torch.empty(max(rms_norm_bwd_workspace_bytes(tokens, dim), 1), dtype=torch.uint8, device=device)


def rms_norm_bwd(dy, s, weight, eps: float = 1e-6, dres=None, grad_s=None, need_grad_weight=False, grad_weight=None,
                 workspace=None, stream=None):
    """Backward of rms_norm_fwd from s (its second result): (grad_s bf16 [T x D], grad_weight fp32 [D] or None).
    grad_s, the gradient of x and of residual alike, includes dres, the gradient that reaches s past the norm;
    grad_s may be dres or dy.  grad_weight is formed where it is given or need_grad_weight."""
    torch = _torch()
    T, D = _rows(s, "s")
    dev = s.device
    chk = _Args(dev)
    chk.bf16(dy, "dy", (T, D))
    chk.bf16(s, "s", (T, D))
    dtype = _norm_weight(weight, chk, D)
    if dres is not None:
        chk.bf16(dres, "dres", (T, D))
    if grad_s is not None:
        chk.bf16(grad_s, "grad_s", (T, D))
    need_grad_weight = need_grad_weight or grad_weight is not None
    if grad_weight is not None:
        chk.f32(grad_weight, "grad_weight", (D,))
    chk.done()
    handle = _stream_on(dev, stream)
    wsb = 0
    with _alloc_on(stream):
        if grad_s is None:
            grad_s = _bf16_like(s)
        if need_grad_weight:
            if grad_weight is None:
                grad_weight = torch.empty(D, dtype=torch.float32, device=dev)
            if workspace is None:
                workspace = rms_norm_bwd_workspace(T, D, dev)
                wsb = workspace.numel()
            else:
                wsb = _workspace(workspace, dev, lambda: rms_norm_bwd_workspace_bytes(T, D))
    _check(lib().qlora_rms_norm_bwd(dy.data_ptr(), s.data_ptr(), _ptr(dres), T, D, weight.data_ptr(), dtype, float(eps),
                                    grad_s.data_ptr(), _ptr(grad_weight), _ptr(workspace) if wsb else None, wsb, handle),
           "qlora_rms_norm_bwd")
    return grad_s, grad_weight


def gated_act_fwd(gate, up, activation: str = "silu", h=None, need_h=True, act8: Act8 = None, need_act8=False,
                  stream=None):
    """The gated product alone: (h, act8) with h = bf16(act(gate) up) [T x N], N % 64 == 0, and its 8-bit checkpoint
    where it is given or need_act8 (h is None with need_h=False).  activation: "silu" or "gelu_tanh".  h may be gate
    or up."""
    code = _activation(activation)
    T, N = _rows(gate, "gate")
    dev = gate.device
    chk = _Args(dev)
    chk.bf16(gate, "gate", (T, N))
    chk.bf16(up, "up", (T, N))
    need_act8 = need_act8 or act8 is not None
    if not need_h:
        h = None
        if not need_act8:
            raise ValueError("need_h=False needs an 8-bit result")
    elif h is not None:
        chk.bf16(h, "h", (T, N))
    _out8(act8, T, N, chk)
    chk.done()
    handle = _stream_on(dev, stream)
    with _alloc_on(stream):
        if need_h and h is None:
            h = _bf16_like(gate)
        if need_act8 and act8 is None:
            act8 = Act8.empty(T, N, dev)
    _check(lib().qlora_gated_act_fwd(gate.data_ptr(), up.data_ptr(), T, N, code, _ptr(h), _ref8(act8), handle),
           "qlora_gated_act_fwd")
    return h, act8


def gated_act_bwd(dh, gate, up, activation: str = "silu", dgate=None, dup=None, stream=None):
    """Backward of the gated product: (dgate, dup) = (bf16(dh up act'(gate)), bf16(dh act(gate))), which
    linear_set_bwd, linear_set_bwd_act8 and linear_bwd_dropout take as the projections' dy.  dgate and dup may
    each be any one of dh, gate and up, but not both the same."""
    code = _activation(activation)
    T, N = _rows(gate, "gate")
    dev = gate.device
    chk = _Args(dev)
    chk.bf16(dh, "dh", (T, N))
    chk.bf16(gate, "gate", (T, N))
    chk.bf16(up, "up", (T, N))
    if dgate is not None:
        chk.bf16(dgate, "dgate", (T, N))
    if dup is not None:
        chk.bf16(dup, "dup", (T, N))
    chk.done()
    handle = _stream_on(dev, stream)
    with _alloc_on(stream):
        if dgate is None:
            dgate = _bf16_like(gate)
        if dup is None:
            dup = _bf16_like(gate)
    _check(lib().qlora_gated_act_bwd(dh.data_ptr(), gate.data_ptr(), up.data_ptr(), T, N, code, dgate.data_ptr(),
                                     dup.data_ptr(), handle), "qlora_gated_act_bwd")
    return dgate, dup


class Gated(NamedTuple):
    """Results of linear_gated_fwd; None where a call was not asked for one."""
    h: "object"
    act8: "Act8"
    gate: "object"
    up: "object"
    u: "object"


@functools.lru_cache(maxsize=1024)
def linear_gated_workspace_bytes(tokens: int, n_ff: int, n_in: int, r: int) -> int:
    return int(lib().qlora_linear_gated_workspace_bytes(tokens, n_ff, n_in, r))


def linear_gated_workspace(tokens: int, n_ff: int, n_in: int, r: int, device="cuda"):
    """A workspace for linear_gated_fwd of exactly these sizes (reusable by successive calls on one stream; fewer
    tokens may need more)."""
    torch = _torch()
    return torch.empty(max(linear_gated_workspace_bytes(tokens, n_ff, n_in, r), 1), dtype=torch.uint8, device=device)


def linear_gated_fwd(x, qs, A_set, Bs, scale: float, activation: str = "silu", keep=True, h=None, need_h=True,
                     act8: Act8 = None, need_act8=False, gate=None, up=None, u_out=None, workspace=None,
                     stream=None) -> Gated:
    """The gated product of a feed-forward block behind its projections: h = bf16(act(gate) up) with gate and up the
    linear_set_fwd of qs = [gate, up] (both [n_ff x n_in], n_ff % 64 == 0), taken in fp32; u = x A_set^T is rounded to
    bf16, as it is returned, before it meets B.  keep: gate, up and u, which the backward pass reads (gated_act_bwd, then
    linear_set_bwd or linear_set_bwd_act8), are returned too.  act8: h's 8-bit
    checkpoint, where it is given or need_act8; need_h=False leaves out h itself."""
    torch = _torch()
    code = _activation(activation)
    if len(qs) != 2:
        raise ValueError(f"qs must hold the gate and the up weight, not {len(qs)}")
    T, count, r, dev, chk = _set_dims(x, qs, A_set)
    N, K = qs[0].n_out, qs[0].n_in
    if qs[1].n_out != N:
        raise ValueError(f"up has n_out {qs[1].n_out}, gate has {N}")
    if N % 64:
        raise ValueError(f"n_out must be a multiple of 64, not {N}")
    _check_list(Bs, 2, "Bs")
    chk.bf16(Bs[0], "Bs[0]", (N, r))
    chk.bf16(Bs[1], "Bs[1]", (N, r))
    need_act8 = need_act8 or act8 is not None
    if not need_h:
        h = None
        if not need_act8:
            raise ValueError("need_h=False needs an 8-bit result")
    elif h is not None:
        chk.bf16(h, "h", (T, N))
    _out8(act8, T, N, chk)
    if not keep and (gate is not None or up is not None):
        raise ValueError("gate and up are written with keep=True")
    if gate is not None:
        chk.bf16(gate, "gate", (T, N))
    if up is not None:
        chk.bf16(up, "up", (T, N))
    if u_out is not None:
        chk.bf16(u_out, "u_out", (T, 2 * r))
    chk.done()
    handle = _stream_on(dev, stream)
    with _alloc_on(stream):
        bf16 = torch.bfloat16
        if need_h and h is None:
            h = torch.empty((T, N), dtype=bf16, device=dev)
        if need_act8 and act8 is None:
            act8 = Act8.empty(T, N, dev)
        if keep:
            if gate is None:
                gate = torch.empty((T, N), dtype=bf16, device=dev)
            if up is None:
                up = torch.empty((T, N), dtype=bf16, device=dev)
            if u_out is None:
                u_out = torch.empty((T, 2 * r), dtype=bf16, device=dev)
        if workspace is None:
            ws = linear_gated_workspace(T, N, K, r, dev)
            wsb = ws.numel()
        else:
            ws = workspace
            wsb = _workspace(ws, dev, lambda: linear_gated_workspace_bytes(T, N, K, r))
    st = (NF4WeightStruct * 2)(qs[0].struct(), qs[1].struct())
    _check(lib().qlora_linear_gated_fwd(_ptr(x), T, st, _ptr(A_set), _ptrs(Bs), r, float(scale), code, _ptr(h),
                                        _ref8(act8), _ptr(gate), _ptr(up), _ptr(u_out), _ptr(ws), wsb, handle),
           "qlora_linear_gated_fwd")
    return Gated(h, act8, gate, up, u_out)
