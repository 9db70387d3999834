"""Python binding of the gfx950 block-scaled FP4 library (libfp4.so).

Argument marshalling only: every step of quantize, dequantize and the GEMMs
runs in the HIP kernels behind the C ABI of include/fp4.h.  torch provides
device memory and the current stream.  There is no fallback: if libfp4.so is
missing or fails to load, every call raises.

Names follow the C ABI: fp4_quantize, fp4_quantize_transposed, fp4_quantize_both, fp4_dequantize, fp4_gemm, fp4_wo_gemm,
fp4_wo_gemm_lora, fp4_lora_apply, fp4_lora_backward, fp4_token_logprobs, fp4_token_logprobs_backward,
fp4_residual_norm, fp4_residual_norm_backward, plus the amax state (per-tensor maximum refreshed every N calls,
ue5m3-fp4-pretraining "Что сделали").
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4.so")

SCALE_FORMATS = {"e4m3": 0, "ue5m3": 1, "e3m4": 2, "e1m6": 3, "e8m0": 4, "e2m5": 5, "e5m2": 6, "e6m1": 7,
                 "e7m0": 8}
ROUNDING = {"nearest": 0, "stochastic": 1}
AMAX = {"none": 0, "current": 1, "delayed": 2}
TRANSFORM = {"none": 0, "rht": 1}
ELEMENT = {"e2m1": 0, "int4": 1, "fp8_e4m3": 2, "int8": 3, "fp6_e2m3": 4, "fp6_e3m2": 5, "int6": 6}
ELEMENT_BITS = {"e2m1": 4, "int4": 4, "fp8_e4m3": 8, "int8": 8, "fp6_e2m3": 6, "fp6_e3m2": 6, "int6": 6}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}

FP4_OK = 0


class Fp4Format(ctypes.Structure):
    _fields_ = [("block", ctypes.c_int32), ("scale", ctypes.c_int32), ("rounding", ctypes.c_int32),
                ("amax", ctypes.c_int32), ("transform", ctypes.c_int32), ("transform_signs", ctypes.c_uint32),
                ("element", ctypes.c_int32)]


class Fp4TensorC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("fmt", Fp4Format)]


class Fp4LoraBankC(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("adapters", ctypes.c_int64), ("rank", ctypes.c_int64), ("k", ctypes.c_int64), ("n", ctypes.c_int64)]


class Fp4NormC(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("res", ctypes.c_void_p), ("ld_res", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("w_pre", ctypes.c_void_p),
                ("w_post", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float), ("x_dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32)]


# Fp4NormC's layout; packing it costs a third of filling a ctypes.Structure.
_NORM_ARGS = struct.Struct("@PqPqqqPPPffiii4x")
assert _NORM_ARGS.size == ctypes.sizeof(Fp4NormC)


class Fp4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None


def lib():
    """The loaded libfp4.so (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u64, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_uint32
    f32 = ctypes.c_float
    T, LB = ctypes.POINTER(Fp4TensorC), ctypes.POINTER(Fp4LoraBankC)
    sig = {
        "fp4_version": (i32, []),
        "fp4_status_string": (ctypes.c_char_p, [i32]),
        "fp4_amax_state_create": (i32, [u32, ctypes.POINTER(vp)]),
        "fp4_amax_state_destroy": (i32, [vp]),
        "fp4_amax_state_get": (i32, [vp, ctypes.POINTER(u64), ctypes.POINTER(ctypes.c_float)]),
        "fp4_amax_state_set": (i32, [vp, u64, ctypes.c_float]),
        "fp4_amax_state_fallbacks": (i32, [vp, ctypes.POINTER(u32)]),
        "fp4_set_exchange_wait": (i32, [u64, ctypes.POINTER(u64)]),
        "fp4_set_gemm_small_outputs": (i32, [i64, ctypes.POINTER(i64)]),
        "fp4_quantize": (i32, [vp, i32, i64, T, vp, u64, u64, vp]),
        "fp4_quantize_noalloc": (i32, [vp, i32, i64, T, u64, u64, vp]),
        "fp4_quantize_transposed": (i32, [vp, i32, i64, T, vp, u64, u64, vp]),
        "fp4_quantize_both": (i32, [vp, i32, i64, T, T, vp, u64, u64, vp]),
        "fp4_dequantize": (i32, [T, vp, i32, i64, vp]),
        "fp4_gemm": (i32, [T, T, vp, i64, vp]),
        "fp4_wo_gemm": (i32, [vp, i64, i64, T, vp, i64, vp]),
        "fp4_lora_workspace": (i64, [i32, i64, i64, i64, i64, i64]),
        "fp4_lora_apply": (i32, [vp, i64, i64, LB, vp, vp, i64, vp, i64, vp, vp, i64, vp]),
        "fp4_lora_backward": (i32, [vp, i64, vp, i64, i64, vp, LB, vp, vp, i64, vp, i64, vp, vp, i32, vp, i64, vp]),
        "fp4_wo_gemm_lora": (i32, [vp, i64, i64, T, LB, vp, vp, i64, vp, i64, vp]),
        "fp4_token_logprobs_workspace": (i64, [i64, i64, i32]),
        "fp4_token_logprobs": (i32, [vp, i32, i64, i64, i64, vp, f32, i32, vp, vp, vp, vp, vp, vp, i64, vp]),
        "fp4_token_logprobs_backward": (i32, [vp, i32, i64, i64, i64, vp, f32, vp, vp, vp, vp, vp, i64, vp]),
        "fp4_residual_norm": (i32, [vp, vp, i64, vp, i64, vp, vp]),
        "fp4_residual_norm_workspace": (i64, [i64, i64, i32]),
        "fp4_residual_norm_backward": (i32, [vp, vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().fp4_status_string(status).decode()


def _check(status: int, what: str):
    if status != FP4_OK:
        raise Fp4Error(status, what)


# The handle of a device's current stream: torch's private call for it makes no
# Stream object, whose cost a launch-bound call notices.
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream, device: torch.device | None = None) -> int:
    if stream is None:
        return _current_handle(torch.cuda.current_device() if device is None else device.index)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on_device(what: str, *tensors: torch.Tensor) -> torch.device:
    """Every tensor a call hands to the library must be a CUDA tensor, all on
    one device (the kernels dereference these pointers on that device)."""
    dev = None
    for t in tensors:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{what}: every tensor must be a CUDA tensor")
        if dev is None:
            dev, index = t.device, t.get_device()
        elif t.get_device() != index:
            raise ValueError(f"{what}: tensors on different devices ({dev} and {t.device})")
    return dev


def _check_dense_out(out: torch.Tensor, shape: tuple, dtypes: tuple, what: str):
    """An output the kernels write row by row through (pointer, row stride):
    exactly the shape, one of the dtypes and unit column stride."""
    if tuple(out.shape) != tuple(shape) or out.dtype not in dtypes or (out.dim() == 2 and out.numel() != 0
                                                                         and out.stride(1) != 1):
        raise ValueError(f"{what}: out must be {list(shape)} with unit column stride and dtype in {dtypes}")


# ---------------------------------------------------------------------------
@dataclass
class QTensor:
    """A quantized tensor: codes [rows, cols/2] (low nibble = even element),
    scales [rows, cols/block], tensor_scale [2] = {g, amax used}; transform
    "rht" with rht_signs marks a blockwise randomized Hadamard transform
    applied before quantization."""
    q: torch.Tensor
    scales: torch.Tensor
    tensor_scale: torch.Tensor
    rows: int
    cols: int
    block: int
    scale: str
    rounding: str = "nearest"
    amax: str = "current"
    transform: str = "none"
    rht_signs: int = 0
    element: str = "e2m1"

    @classmethod
    def empty(cls, rows: int, cols: int, block: int, scale: str, rounding: str = "nearest",
              amax: str = "current", device="cuda", transform: str = "none", rht_signs: int = 0,
              element: str = "e2m1"):
        q = torch.empty((rows, cols * ELEMENT_BITS[element] // 8), dtype=torch.uint8, device=device)
        s = torch.empty((rows, cols // block), dtype=torch.uint8, device=device)
        ts = torch.empty(2, dtype=torch.float32, device=device)
        return cls(q, s, ts, rows, cols, block, scale, rounding, amax, transform, rht_signs, element)

    def c(self) -> Fp4TensorC:
        # the library reads or writes rows * cols * bits / 8 code bytes and
        # rows * cols / block scale bytes through these pointers, densely
        qb = self.rows * (self.cols * ELEMENT_BITS[self.element] // 8)
        if not (self.q.is_contiguous() and self.scales.is_contiguous() and self.tensor_scale.is_contiguous()):
            raise ValueError("QTensor buffers must be contiguous")
        if self.q.numel() * self.q.element_size() < qb or \
                self.scales.numel() * self.scales.element_size() < self.rows * (self.cols // self.block) or \
                self.tensor_scale.numel() < 2:
            raise ValueError(f"QTensor buffers are smaller than a [{self.rows}, {self.cols}] tensor on the "
                             f"{self.element} grid needs")
        fmt = Fp4Format(self.block, SCALE_FORMATS[self.scale], ROUNDING[self.rounding], AMAX[self.amax],
                        TRANSFORM[self.transform], self.rht_signs & 0xFFFFFFFF, ELEMENT[self.element])
        return Fp4TensorC(self.q.data_ptr(), self.scales.data_ptr(), self.tensor_scale.data_ptr(),
                          self.rows, self.cols, fmt)


class AmaxState:
    """Per-tensor amax state: refreshed every `interval` calls (CURRENT uses
    it too, refreshing on every call).  Owns 17664 bytes of device memory."""

    def __init__(self, interval: int = 50):
        h = ctypes.c_void_p()
        _check(lib().fp4_amax_state_create(interval, ctypes.byref(h)), "fp4_amax_state_create")
        self._h = h
        self.interval = interval

    @property
    def handle(self):
        return self._h

    def get(self):
        calls, amax = ctypes.c_uint64(), ctypes.c_float()
        _check(lib().fp4_amax_state_get(self._h, ctypes.byref(calls), ctypes.byref(amax)), "fp4_amax_state_get")
        return calls.value, amax.value

    def set(self, calls: int, amax: float):
        _check(lib().fp4_amax_state_set(self._h, calls, amax), "fp4_amax_state_set")

    def fallbacks(self) -> int:
        """Workgroups of single-pass refreshes on this state that gave up
        waiting for the others and read the whole tensor themselves."""
        n = ctypes.c_uint32()
        _check(lib().fp4_amax_state_fallbacks(self._h, ctypes.byref(n)), "fp4_amax_state_fallbacks")
        return n.value

    def close(self):
        if self._h is not None and self._h.value:
            lib().fp4_amax_state_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def set_exchange_wait(ticks: int) -> int:
    """Set the process-wide bound on a single-pass refresh's wait for the
    other workgroups (ticks of the 100 MHz device clock); returns the
    previous bound."""
    prev = ctypes.c_uint64()
    _check(lib().fp4_set_exchange_wait(ticks, ctypes.byref(prev)), "fp4_set_exchange_wait")
    return prev.value


def set_gemm_small_outputs(outputs: int) -> int:
    """Set the process-wide bound on M * N up to which fp4_gemm takes the
    one-wave-per-32x32-tile path for the pairings it covers (E8M0 operands:
    an eighth of it; 0 turns the path off); returns the previous bound."""
    prev = ctypes.c_int64()
    _check(lib().fp4_set_gemm_small_outputs(outputs, ctypes.byref(prev)), "fp4_set_gemm_small_outputs")
    return prev.value


# One amax workspace per (device, stream) for calls with the current policy
# that bring no state: calls on one stream run in order, so they can share
# it, and no call allocates.
_default_states: dict = {}


def _default_state(device: torch.device, stream_handle: int) -> AmaxState:
    key = (device.index, stream_handle)
    st = _default_states.get(key)
    if st is None:
        with torch.cuda.device(device):
            st = AmaxState(1)
        _default_states[key] = st
    return st


def _resolve_state(amax: str, state: AmaxState | None, device: torch.device, stream_handle: int):
    if amax == "none" or state is not None:
        return state
    if amax == "delayed":
        raise ValueError("the delayed amax policy needs an AmaxState")
    return _default_state(device, stream_handle)


def _check_out(t: QTensor, rows: int, cols: int, block: int, element: str):
    """A caller-provided output must hold the codes and scales of a [rows,
    cols] tensor on `element` (the kernels write exactly that many bytes)."""
    qb = cols * ELEMENT_BITS[element] // 8
    if (t.rows, t.cols) != (rows, cols) or t.q.numel() < rows * qb or t.scales.numel() < rows * (cols // block) \
            or t.tensor_scale.numel() < 2 or not (t.q.is_contiguous() and t.scales.is_contiguous()):
        raise ValueError(f"out does not hold a [{rows}, {cols}] tensor on the {element} grid with block {block}")


def fp4_quantize(x: torch.Tensor, block: int = 16, scale: str = "e4m3", rounding: str = "nearest",
                 amax: str = "current", state: AmaxState | None = None, seed: int = 0, offset: int = 0,
                 out: QTensor | None = None, stream=None, rht_signs: int | None = None,
                 element: str = "e2m1") -> QTensor:
    """Quantize a 2-D fp32/bf16 CUDA tensor (rows may be strided: x.stride(1)
    must be 1).  DELAYED needs an AmaxState; CURRENT without one uses a
    workspace shared by the calls on the same device and stream.  rht_signs (32-bit sign mask) applies the
    blockwise randomized Hadamard transform before quantization; element
    selects the grid: "e2m1" (default), "int4" (-7..7), the one-byte
    "fp8_e4m3" and "int8" (-127..127), or the six-bit "fp6_e2m3",
    "fp6_e3m2" and "int6" (-31..31)."""
    if x.dim() != 2 or (x.stride(1) != 1 and x.numel() != 0):
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype not in DTYPE:
        raise ValueError("x must be float32 or bfloat16")
    _on_device("fp4_quantize", x, *(() if out is None else (out.q, out.scales, out.tensor_scale)))
    rows, cols = x.shape
    if out is None:
        out = QTensor.empty(rows, cols, block, scale, rounding, amax, device=x.device, element=element)
    else:
        _check_out(out, rows, cols, block, element)
        out.block, out.scale, out.rounding, out.amax = block, scale, rounding, amax
    out.transform, out.rht_signs = ("none", 0) if rht_signs is None else ("rht", rht_signs & 0xFFFFFFFF)
    out.element = element
    sh = _stream(stream, x.device)
    state = _resolve_state(amax, state, x.device, sh)
    out._state = state        # keep the state alive while work is queued
    tc = out.c()
    st = lib().fp4_quantize(x.data_ptr(), DTYPE[x.dtype], x.stride(0), ctypes.byref(tc),
                            state.handle if state is not None else None, seed, offset, sh)
    _check(st, "fp4_quantize")
    return out


def fp4_quantize_noalloc(x: torch.Tensor, out: QTensor, block: int = 16, scale: str = "e4m3",
                         rounding: str = "nearest", amax: str = "current", seed: int = 0, offset: int = 0,
                         stream=None, rht_signs: int | None = None, element: str = "e2m1") -> QTensor:
    """fp4_quantize into a caller-provided output with no allocation: the
    current-amax workspace is the library's static per-device array (calls
    that overlap on one device must be ordered by the caller).  Policies
    "none" and "current"."""
    if x.dim() != 2 or (x.stride(1) != 1 and x.numel() != 0):
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype not in DTYPE:
        raise ValueError("x must be float32 or bfloat16")
    _on_device("fp4_quantize_noalloc", x, out.q, out.scales, out.tensor_scale)
    rows, cols = x.shape
    _check_out(out, rows, cols, block, element)
    out.block, out.scale, out.rounding, out.amax, out.element = block, scale, rounding, amax, element
    out.transform, out.rht_signs = ("none", 0) if rht_signs is None else ("rht", rht_signs & 0xFFFFFFFF)
    tc = out.c()
    _check(lib().fp4_quantize_noalloc(x.data_ptr(), DTYPE[x.dtype], x.stride(0), ctypes.byref(tc), seed, offset,
                                      _stream(stream, x.device)), "fp4_quantize_noalloc")
    return out


def fp4_quantize_transposed(x: torch.Tensor, block: int = 16, scale: str = "e4m3", rounding: str = "nearest",
                            amax: str = "current", state: AmaxState | None = None, seed: int = 0, offset: int = 0,
                            out: QTensor | None = None, stream=None, element: str = "e2m1",
                            rht_signs: int | None = None) -> QTensor:
    """Column-wise quantization of a 2-D fp32/bf16 CUDA tensor x [R, C]: the
    result is the quantized x^T [C, R] (blocks run down the columns of x)."""
    if x.dim() != 2 or (x.stride(1) != 1 and x.numel() != 0):
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype not in DTYPE:
        raise ValueError("x must be float32 or bfloat16")
    _on_device("fp4_quantize_transposed", x, *(() if out is None else (out.q, out.scales, out.tensor_scale)))
    r, c = x.shape
    if out is None:
        out = QTensor.empty(c, r, block, scale, rounding, amax, device=x.device, element=element)
    else:
        _check_out(out, c, r, block, element)
        out.block, out.scale, out.rounding, out.amax = block, scale, rounding, amax
    out.element = element
    out.transform, out.rht_signs = ("none", 0) if rht_signs is None else ("rht", rht_signs & 0xFFFFFFFF)
    sh = _stream(stream, x.device)
    state = _resolve_state(amax, state, x.device, sh)
    out._state = state
    tc = out.c()
    st = lib().fp4_quantize_transposed(x.data_ptr(), DTYPE[x.dtype], x.stride(0), ctypes.byref(tc),
                                       state.handle if state is not None else None, seed, offset, sh)
    _check(st, "fp4_quantize_transposed")
    return out


def fp4_quantize_both(x: torch.Tensor, block: int = 16, scale: str = "e4m3", rounding: str = "nearest",
                      amax: str = "current", state: AmaxState | None = None, seed: int = 0, offset: int = 0,
                      out: tuple | None = None, stream=None, element: str = "e2m1"):
    """Row-wise and column-wise quantization of x [R, C] from one read:
    returns (rowwise [R, C], colwise [C, R]) QTensors, each identical to the
    corresponding single-orientation call."""
    if x.dim() != 2 or (x.stride(1) != 1 and x.numel() != 0):
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype not in DTYPE:
        raise ValueError("x must be float32 or bfloat16")
    r, c = x.shape
    if out is None:
        out = (QTensor.empty(r, c, block, scale, rounding, amax, device=x.device, element=element),
               QTensor.empty(c, r, block, scale, rounding, amax, device=x.device, element=element))
    qr, qc = out
    _on_device("fp4_quantize_both", x, qr.q, qr.scales, qr.tensor_scale, qc.q, qc.scales, qc.tensor_scale)
    _check_out(qr, r, c, block, element)
    _check_out(qc, c, r, block, element)
    for t in (qr, qc):
        t.block, t.scale, t.rounding, t.amax, t.element = block, scale, rounding, amax, element
        t.transform, t.rht_signs = "none", 0
    sh = _stream(stream, x.device)
    state = _resolve_state(amax, state, x.device, sh)
    qr._state = qc._state = state
    tr, tcw = qr.c(), qc.c()
    st = lib().fp4_quantize_both(x.data_ptr(), DTYPE[x.dtype], x.stride(0), ctypes.byref(tr), ctypes.byref(tcw),
                                 state.handle if state is not None else None, seed, offset, sh)
    _check(st, "fp4_quantize_both")
    return qr, qc


def fp4_dequantize(t: QTensor, dtype=torch.float32, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    dev = _on_device("fp4_dequantize", t.q, t.scales, t.tensor_scale, *(() if out is None else (out,)))
    if out is None:
        out = torch.empty((t.rows, t.cols), dtype=dtype, device=dev)
    _check_dense_out(out, (t.rows, t.cols), (torch.float32, torch.bfloat16), "fp4_dequantize")
    tc = t.c()
    _check(lib().fp4_dequantize(ctypes.byref(tc), out.data_ptr(), DTYPE[out.dtype], out.stride(0),
                                _stream(stream, dev)), "fp4_dequantize")
    return out


def fp4_gemm(a: QTensor, b: QTensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """C[M, N] = A[M, K] @ W[N, K]^T in bf16 (fp32 accumulation)."""
    dev = _on_device("fp4_gemm", a.q, a.scales, a.tensor_scale, b.q, b.scales, b.tensor_scale,
                     *(() if out is None else (out,)))
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=dev)
    _check_dense_out(out, (a.rows, b.rows), (torch.bfloat16,), "fp4_gemm")
    ta, tb = a.c(), b.c()
    _check(lib().fp4_gemm(ctypes.byref(ta), ctypes.byref(tb), out.data_ptr(), out.stride(0), _stream(stream, dev)),
           "fp4_gemm")
    return out


def fp4_wo_gemm(x: torch.Tensor, w: QTensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y[M, N] = X[M, K] (bf16) @ W[N, K]^T with W quantized (bf16 out)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or (x.stride(1) != 1 and x.numel() != 0):
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    if x.shape[1] != w.cols:
        raise ValueError(f"x has {x.shape[1]} columns, the weight {w.cols}")
    dev = _on_device("fp4_wo_gemm", x, w.q, w.scales, w.tensor_scale, *(() if out is None else (out,)))
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, w.rows), dtype=torch.bfloat16, device=dev)
    _check_dense_out(out, (m, w.rows), (torch.bfloat16,), "fp4_wo_gemm")
    tw = w.c()
    _check(lib().fp4_wo_gemm(x.data_ptr(), x.stride(0), m, ctypes.byref(tw), out.data_ptr(), out.stride(0),
                             _stream(stream, dev)), "fp4_wo_gemm")
    return out


# ---------------------------------------------------------------------------
# Training and serving of low-rank adapters over quantized weights.  Outputs
# and workspaces that these calls allocate belong to the call's stream, so
# that memory freed here is not handed to another stream's work while the
# call is still queued.
# ---------------------------------------------------------------------------
_LORA_APPLY, _LORA_BACKWARD, _LORA_WO_GEMM = range(3)


_HERE_AND_NOW = contextlib.nullcontext()


def _allocating(stream, device: torch.device):
    if stream is None:
        return _HERE_AND_NOW
    if not isinstance(stream, torch.cuda.Stream):
        # torch takes a pointer of 0 for none given and would make a new stream
        stream = torch.cuda.ExternalStream(int(stream), device) if int(stream) else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _space(nbytes: int, device: torch.device, what: str) -> torch.Tensor | None:
    """A workspace of `nbytes` (a negative number is a status)."""
    if nbytes < 0:
        _check(nbytes, what)
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _is_rows(t, cols: int | None = None, rows: int | None = None) -> bool:
    """A 2-D tensor whose rows are dense."""
    return (t.dim() == 2 and (t.stride(1) == 1 or t.numel() == 0 or t.shape[1] == 1)
            and (cols is None or t.shape[1] == cols) and (rows is None or t.shape[0] == rows))


def _ld(t: torch.Tensor) -> int:
    """Row stride; a single row's is its length, whatever torch keeps there."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _is_vector(t, n: int, dtype: torch.dtype) -> bool:
    return t.dim() == 1 and t.shape[0] == n and t.dtype == dtype and (n < 2 or t.stride(0) == 1)


@dataclass
class LoraBank:
    """Low-rank adapters of one projection: a [adapters, rank, K] and b
    [adapters, N, rank] in bf16, scale [adapters] in fp32.  rank is a multiple
    of 8 up to 128 (pad a smaller one with zeros)."""
    a: torch.Tensor
    b: torch.Tensor
    scale: torch.Tensor

    def c(self) -> Fp4LoraBankC:
        a, b, s = self.a, self.b, self.scale
        if a.dim() != 3 or b.dim() != 3 or s.dim() != 1 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2] \
                or s.shape[0] != a.shape[0]:
            raise ValueError("LoraBank: a is [adapters, rank, K], b is [adapters, N, rank], scale is [adapters]")
        if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16 or s.dtype != torch.float32:
            raise ValueError("LoraBank: a and b must be bfloat16, scale float32")
        if not (a.is_contiguous() and b.is_contiguous() and s.is_contiguous()):
            raise ValueError("LoraBank buffers must be contiguous")
        return Fp4LoraBankC(a.data_ptr(), b.data_ptr(), s.data_ptr(), a.shape[0], a.shape[1], a.shape[2], b.shape[1])


def _lora_rows(what: str, x: torch.Tensor, slots: torch.Tensor, k: int):
    if x.dtype != torch.bfloat16 or not _is_rows(x, k):
        raise ValueError(f"{what}: expected a bf16 [rows, {k}] tensor with unit column stride")
    if not _is_vector(slots, x.shape[0], torch.int32):
        raise ValueError(f"{what}: slots must be int32 [{x.shape[0]}], one adapter (or -1) for each row")


def fp4_wo_gemm_lora(x: torch.Tensor, w: QTensor, bank: LoraBank, slots: torch.Tensor,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp4_wo_gemm plus each row's adapter: Y = X W^T + s_l (X A_l^T) B_l^T
    with l = slots[row] (outside the bank: none), for at most 16 rows."""
    _lora_rows("fp4_wo_gemm_lora", x, slots, w.cols)
    dev = _on_device("fp4_wo_gemm_lora", x, w.q, w.scales, w.tensor_scale, bank.a, bank.b, bank.scale, slots,
                     *(() if out is None else (out,)))
    m, n, L = x.shape[0], w.rows, lib()
    tw, tb = w.c(), bank.c()
    with _allocating(stream, dev):
        if out is None:
            out = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
        else:
            _check_dense_out(out, (m, n), (torch.bfloat16,), "fp4_wo_gemm_lora")
        ws = _space(L.fp4_lora_workspace(_LORA_WO_GEMM, m, tb.n, tb.k, tb.rank, tb.adapters), dev, "fp4_wo_gemm_lora")
        st = L.fp4_wo_gemm_lora(x.data_ptr(), _ld(x), m, ctypes.byref(tw), ctypes.byref(tb), slots.data_ptr(),
                                out.data_ptr(), _ld(out), _ptr(ws), 0 if ws is None else ws.numel(),
                                _stream(stream, dev))
    _check(st, "fp4_wo_gemm_lora")
    return out


def fp4_lora_apply(x: torch.Tensor, bank: LoraBank, slots: torch.Tensor, base: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, stream=None) -> tuple:
    """(y, t): y = base + s_l (x A_l^T) B_l^T for each row's adapter l =
    slots[row], and t = x A_l^T (fp32 [rows, rank]), which fp4_lora_backward
    takes.  base is the shared projection's output (None: zero); out may be
    base."""
    tb = bank.c()
    _lora_rows("fp4_lora_apply", x, slots, tb.k)
    m = x.shape[0]
    dev = _on_device("fp4_lora_apply", x, bank.a, bank.b, bank.scale, slots,
                     *(t for t in (base, out) if t is not None))
    if base is not None:
        _check_dense_out(base, (m, tb.n), (torch.bfloat16,), "fp4_lora_apply: base")
    L = lib()
    with _allocating(stream, dev):
        if out is None:
            out = torch.empty((m, tb.n), dtype=torch.bfloat16, device=dev)
        else:
            _check_dense_out(out, (m, tb.n), (torch.bfloat16,), "fp4_lora_apply")
        t = torch.empty((m, tb.rank), dtype=torch.float32, device=dev)
        ws = _space(L.fp4_lora_workspace(_LORA_APPLY, m, tb.n, tb.k, tb.rank, tb.adapters), dev, "fp4_lora_apply")
        st = L.fp4_lora_apply(x.data_ptr(), _ld(x), m, ctypes.byref(tb), slots.data_ptr(), _ptr(base),
                              0 if base is None else _ld(base), out.data_ptr(), _ld(out), t.data_ptr(), _ptr(ws),
                              0 if ws is None else ws.numel(), _stream(stream, dev))
    _check(st, "fp4_lora_apply")
    return out, t


def fp4_lora_backward(dy: torch.Tensor, x: torch.Tensor, t: torch.Tensor, bank: LoraBank, slots: torch.Tensor,
                      dx_base: torch.Tensor | None = None, grad_dtype=torch.float32, dx: torch.Tensor | None = None,
                      stream=None) -> tuple:
    """(dx, da, db) of fp4_lora_apply for the gradient dy [rows, N] of its y.
    t is fp4_lora_apply's; dx_base the gradient that reaches x through the
    shared projection (None: zero; dx may be dx_base); da and db have the
    bank's shapes in grad_dtype."""
    tb = bank.c()
    _lora_rows("fp4_lora_backward", x, slots, tb.k)
    m = x.shape[0]
    if dy.dtype != torch.bfloat16 or not _is_rows(dy, tb.n, m):
        raise ValueError(f"fp4_lora_backward: dy must be bf16 [{m}, {tb.n}] with unit column stride")
    if t.dtype != torch.float32 or tuple(t.shape) != (m, tb.rank) or not t.is_contiguous():
        raise ValueError(f"fp4_lora_backward: t must be the dense fp32 [{m}, {tb.rank}] of fp4_lora_apply")
    if grad_dtype not in DTYPE:
        raise ValueError("fp4_lora_backward: grad_dtype must be float32 or bfloat16")
    dev = _on_device("fp4_lora_backward", dy, x, t, bank.a, bank.b, bank.scale, slots,
                     *(v for v in (dx_base, dx) if v is not None))
    if dx_base is not None:
        _check_dense_out(dx_base, (m, tb.k), (torch.bfloat16,), "fp4_lora_backward: dx_base")
    L = lib()
    with _allocating(stream, dev):
        if dx is None:
            dx = _empty_as(x)
        else:
            _check_dense_out(dx, (m, tb.k), (torch.bfloat16,), "fp4_lora_backward")
        da = torch.empty(bank.a.shape, dtype=grad_dtype, device=dev)
        db = torch.empty(bank.b.shape, dtype=grad_dtype, device=dev)
        ws = _space(L.fp4_lora_workspace(_LORA_BACKWARD, m, tb.n, tb.k, tb.rank, tb.adapters), dev, "fp4_lora_backward")
        st = L.fp4_lora_backward(dy.data_ptr(), _ld(dy), x.data_ptr(), _ld(x), m, t.data_ptr(), ctypes.byref(tb),
                                 slots.data_ptr(), _ptr(dx_base), 0 if dx_base is None else _ld(dx_base),
                                 dx.data_ptr(), _ld(dx), da.data_ptr(), db.data_ptr(), DTYPE[grad_dtype], _ptr(ws),
                                 0 if ws is None else ws.numel(), _stream(stream, dev))
    _check(st, "fp4_lora_backward")
    return dx, da, db


@dataclass
class TokenLogprobs:
    """logprob (None without tokens) and entropy [rows]; top_ids (int32) and
    top_logprobs [rows, top], largest first (None for top = 0); stats [rows,
    2] for the backward call."""
    logprob: torch.Tensor | None
    entropy: torch.Tensor
    stats: torch.Tensor
    top_ids: torch.Tensor | None
    top_logprobs: torch.Tensor | None


def _logits(what: str, logits: torch.Tensor, tokens: torch.Tensor | None):
    if logits.dtype not in DTYPE or not _is_rows(logits) or logits.shape[1] < 1:
        raise ValueError(f"{what}: logits must be a float32 or bfloat16 [rows, vocab] tensor with unit column stride")
    if tokens is not None and not _is_vector(tokens, logits.shape[0], torch.int64):
        raise ValueError(f"{what}: tokens must be int64 [{logits.shape[0]}]")


def fp4_token_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, temperature: float = 1.0,
                       top: int = 0, stream=None) -> TokenLogprobs:
    """Log probability of each row's token under softmax(logits /
    temperature) (0 for a token outside the vocabulary, such as -100), the
    entropy, and the `top` (up to 32) most probable tokens."""
    _logits("fp4_token_logprobs", logits, tokens)
    dev = _on_device("fp4_token_logprobs", logits, *(() if tokens is None else (tokens,)))
    n, v = logits.shape
    L = lib()
    with _allocating(stream, dev):
        ws = _space(L.fp4_token_logprobs_workspace(n, v, top), dev, "fp4_token_logprobs")
        logprob = torch.empty(n, dtype=torch.float32, device=dev) if tokens is not None else None
        entropy = torch.empty(n, dtype=torch.float32, device=dev)
        stats = torch.empty((n, 2), dtype=torch.float32, device=dev)
        ids = torch.empty((n, top), dtype=torch.int32, device=dev) if top else None
        best = torch.empty((n, top), dtype=torch.float32, device=dev) if top else None
        st = L.fp4_token_logprobs(logits.data_ptr(), DTYPE[logits.dtype], _ld(logits), n, v, _ptr(tokens), temperature,
                                  top, _ptr(logprob), entropy.data_ptr(), stats.data_ptr(), _ptr(ids), _ptr(best),
                                  _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream, dev))
    _check(st, "fp4_token_logprobs")
    return TokenLogprobs(logprob, entropy, stats, ids, best)


def fp4_token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor | None, saved: TokenLogprobs,
                                grad_logprob: torch.Tensor | None = None, grad_entropy: torch.Tensor | None = None,
                                temperature: float = 1.0, out: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """The gradient of the logits for the gradients of logprob and entropy
    (fp32 [rows]; None: zero).  logits, tokens and temperature are the forward
    call's, saved its result; out may be the logits."""
    what = "fp4_token_logprobs_backward"
    _logits(what, logits, tokens)
    n, v = logits.shape
    for g in (grad_logprob, grad_entropy):
        if g is not None and not _is_vector(g, n, torch.float32):
            raise ValueError(f"{what}: gradients must be float32 [{n}]")
    if grad_logprob is not None and tokens is None:
        raise ValueError(f"{what}: grad_logprob needs the tokens")
    if not _is_vector(saved.entropy, n, torch.float32) or tuple(saved.stats.shape) != (n, 2) \
            or saved.stats.dtype != torch.float32 or not saved.stats.is_contiguous():
        raise ValueError(f"{what}: saved is not the result of a forward call on these logits")
    dev = _on_device(what, logits, saved.entropy, saved.stats,
                     *(t for t in (tokens, grad_logprob, grad_entropy, out) if t is not None))
    with _allocating(stream, dev):
        if out is None:
            out = _empty_as(logits)
        elif out.dtype != logits.dtype or not _is_rows(out, v, n):
            raise ValueError(f"{what}: out must be [{n}, {v}] of the logits' dtype with unit column stride")
        st = lib().fp4_token_logprobs_backward(logits.data_ptr(), DTYPE[logits.dtype], _ld(logits), n, v, _ptr(tokens),
                                               temperature, saved.entropy.data_ptr(), saved.stats.data_ptr(),
                                               _ptr(grad_logprob), _ptr(grad_entropy), out.data_ptr(), _ld(out),
                                               _stream(stream, dev))
    _check(st, what)
    return out


def _norm_args(what: str, x, res, w_pre, w_post, gate, alpha, eps) -> bytes:
    if x.dtype not in DTYPE or not _is_rows(x) or res.dtype not in DTYPE or not _is_rows(res, x.shape[1], x.shape[0]):
        raise ValueError(f"{what}: x and res must be float32 or bfloat16 [rows, cols] tensors with unit column stride")
    m, c = x.shape
    wd = w_pre.dtype
    if wd not in DTYPE or not _is_vector(w_pre, c, wd) or (w_post is not None and not _is_vector(w_post, c, wd)):
        raise ValueError(f"{what}: weights must be dense [{c}] vectors of one dtype, float32 or bfloat16")
    if gate is not None and not _is_vector(gate, m, torch.float32):
        raise ValueError(f"{what}: gate must be float32 [{m}]")
    return _NORM_ARGS.pack(x.data_ptr(), _ld(x), res.data_ptr(), _ld(res), m, c, w_pre.data_ptr(),
                           0 if w_post is None else w_post.data_ptr(), 0 if gate is None else gate.data_ptr(),
                           alpha, eps, DTYPE[x.dtype], DTYPE[res.dtype], DTYPE[wd])


def _empty_as(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def fp4_residual_norm(x: torch.Tensor, res: torch.Tensor, w_pre: torch.Tensor, w_post: torch.Tensor | None = None,
                      gate: torch.Tensor | None = None, alpha: float = 1.0, eps: float = 1e-6, stream=None) -> tuple:
    """(h, n, stats): h = alpha res + gate RMSNorm(x) w_post (x itself without
    w_post; gate fp32 [rows], 1 without) in res' dtype and n = RMSNorm(h)
    w_pre in x's; stats goes to fp4_residual_norm_backward."""
    args = _norm_args("fp4_residual_norm", x, res, w_pre, w_post, gate, alpha, eps)
    dev = _on_device("fp4_residual_norm", x, res, w_pre, *(t for t in (w_post, gate) if t is not None))
    m, c = x.shape
    with _allocating(stream, dev):
        h, n = _empty_as(res), _empty_as(x)
        stats = torch.empty((m, 2), dtype=torch.float32, device=dev)
        st = lib().fp4_residual_norm(args, h.data_ptr(), c, n.data_ptr(), c, stats.data_ptr(),
                                     _stream(stream, dev))
    _check(st, "fp4_residual_norm")
    return h, n, stats


@dataclass
class ResidualNormGrads:
    """dx and dres in the dtypes of x and res; dw_pre, dw_post [cols] and
    dgate [rows] in fp32 (None where the call had no w_post, gate)."""
    dx: torch.Tensor
    dres: torch.Tensor
    dw_pre: torch.Tensor
    dw_post: torch.Tensor | None
    dgate: torch.Tensor | None


def fp4_residual_norm_backward(dn: torch.Tensor | None, dh: torch.Tensor | None, x: torch.Tensor, res: torch.Tensor,
                               w_pre: torch.Tensor, stats: torch.Tensor, w_post: torch.Tensor | None = None,
                               gate: torch.Tensor | None = None, alpha: float = 1.0, stream=None) -> ResidualNormGrads:
    """Gradients of fp4_residual_norm for the gradients dn of n and dh of h
    (None: zero); the other arguments are the forward call's."""
    what = "fp4_residual_norm_backward"
    args = _norm_args(what, x, res, w_pre, w_post, gate, alpha, 0.0)
    m, c = x.shape
    for g, like, name in ((dn, x, "dn"), (dh, res, "dh")):
        if g is not None and (g.dtype != like.dtype or not _is_rows(g, c, m)):
            raise ValueError(f"{what}: {name} must be {like.dtype} [{m}, {c}] with unit column stride")
    if tuple(stats.shape) != (m, 2) or stats.dtype != torch.float32 or not stats.is_contiguous():
        raise ValueError(f"{what}: stats must be the forward call's")
    dev = _on_device(what, x, res, w_pre, stats, *(t for t in (dn, dh, w_post, gate) if t is not None))
    L = lib()
    with _allocating(stream, dev):
        dx, dres = _empty_as(x), _empty_as(res)
        dw_pre = torch.empty(c, dtype=torch.float32, device=dev)
        dw_post = torch.empty(c, dtype=torch.float32, device=dev) if w_post is not None else None
        dgate = _empty_as(gate) if gate is not None else None
        ws = _space(L.fp4_residual_norm_workspace(m, c, w_post is not None), dev, what)
        st = L.fp4_residual_norm_backward(args, stats.data_ptr(), _ptr(dn), 0 if dn is None else _ld(dn),
                                          _ptr(dh), 0 if dh is None else _ld(dh), dx.data_ptr(), c, dres.data_ptr(), c,
                                          dw_pre.data_ptr(), _ptr(dw_post), _ptr(dgate), _ptr(ws),
                                          0 if ws is None else ws.numel(), _stream(stream, dev))
    _check(st, what)
    return ResidualNormGrads(dx, dres, dw_pre, dw_post, dgate)


__all__ = ["fp4_quantize", "fp4_quantize_transposed", "fp4_quantize_both", "fp4_dequantize", "fp4_gemm",
           "fp4_wo_gemm", "AmaxState", "QTensor", "Fp4Error", "SCALE_FORMATS", "lib", "status_string", "LIB_PATH",
           "set_exchange_wait", "set_gemm_small_outputs", "fp4_quantize_noalloc", "LoraBank", "fp4_wo_gemm_lora",
           "fp4_lora_apply", "fp4_lora_backward", "TokenLogprobs", "fp4_token_logprobs",
           "fp4_token_logprobs_backward", "fp4_residual_norm", "ResidualNormGrads", "fp4_residual_norm_backward"]
