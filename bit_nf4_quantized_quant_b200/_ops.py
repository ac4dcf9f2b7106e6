"""Thin binding of libqlora_nf4.so (argument marshalling only).

Every function has the name of the C entry point it calls (see
``include/qlora_nf4.h``) and takes torch tensors for the device buffers, whose
pointers and the current CUDA stream are passed through unchanged.  All
computation happens in the library's CUDA kernels; if the library cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora_nf4.so")

QLORA_OK = 0
QLORA_ERR_NULL = -1
QLORA_ERR_TIMEOUT = -8
QLORA_ERR_VALUE = -9

_lib = None


class QLoRAError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {code} ({status_string(code)})")


QLORA_QUANT_NF4 = 0
QLORA_QUANT_FP4 = 1
QLORA_ACT8_INT8 = 0
QLORA_ACT8_E4M3 = 1
QLORA_ACT8_BLOCK = 32
QLORA_LOGITS_BF16 = 0
QLORA_LOGITS_FP32 = 1
QLORA_PREF_SIGMOID = 0
QLORA_PREF_HINGE = 1
QLORA_PREF_IPO = 2


class _Weight(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("mean", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("quant_type", ctypes.c_int32)]


class _Act8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("M", ctypes.c_int64),
                ("K", ctypes.c_int64), ("fmt", ctypes.c_int32)]


def lib():
    """Load the shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libqlora_nf4.so not found at {LIB_PATH}; run "
                               "`python -m bit_nf4_quantized_quant_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        u64 = ctypes.c_uint64
        WP = ctypes.POINTER(_Weight)
        sig = {
            "nf4_codebook": (i32, [P]),
            "quant4_codebook": (i32, [i32, P]),
            "quant4_quantize_dq": (i32, [P, i64, i64, i32, P, P, P, P, P]),
            "nf4_dequant_merge": (i32, [WP, P, P, i32, f32, P, P]),
            "adamw_8bit_step": (i32, [P, P, i64, P, P, P, P, i64, f32, f32, f32, f32, f32, P]),
            "qlora_dropout_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64, i32]),
            "qlora_linear_fwd_dropout": (i32, [P, i64, WP, P, P, i32, f32, f32, u64, u64, P, P, P,
                                               ctypes.c_size_t, P]),
            "qlora_linear_bwd_dropout": (i32, [P, P, i64, WP, P, P, i32, f32, f32, u64, u64, P, P, P, P, P,
                                               ctypes.c_size_t, P]),
            "nf4dq_sizes": (i32, [i64, i64, P, P, P]),
            "nf4_quantize_dq": (i32, [P, i64, i64, P, P, P, P, P]),
            "nf4_dequant": (i32, [WP, P, P]),
            "qlora_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64, i32]),
            "qlora_linear_fwd": (i32, [P, i64, WP, P, P, i32, f32, P, P, P, ctypes.c_size_t, P]),
            "qlora_linear_bwd": (i32, [P, P, i64, WP, P, P, i32, f32, P, P, P, P, P, ctypes.c_size_t, P]),
            "act8_sizes": (i32, [i64, i64, P, P]),
            "act8_quantize": (i32, [P, i64, i64, i32, P, P, P]),
            "act8_dequant": (i32, [ctypes.POINTER(_Act8), P, P]),
            "qlora_act8_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64, i32, i32]),
            "qlora_linear_bwd_act8": (i32, [ctypes.POINTER(_Act8), P, WP, P, P, i32, f32, f32, u64, u64, P, P, P, P,
                                            P, ctypes.c_size_t, P]),
            "loss_workspace_bytes": (ctypes.c_size_t, [i64]),
            "token_logprob": (i32, [P, i32, i64, i64, i64, f32, P, P, P]),
            "preference_loss": (i32, [P, i32, i64, i64, i64, f32, P, P, i64, P, i32, f32, f32, f32, i32, f32, P, P,
                                      P, P, i64, P, ctypes.c_size_t, P]),
            "policy_loss": (i32, [P, i32, i64, i64, i64, f32, P, P, P, P, P, f32, f32, f32, f32, P, P, P, i64, P,
                                  ctypes.c_size_t, P]),
            "qlora_status_string": (ctypes.c_char_p, [i32]),
            "qlora_device_status": (i32, [i32]),
            "qlora_last_path": (i32, []),
            "qlora_pair_schedule": (i32, [i64, i64, i32, i32, P, P, P]),
            "qlora_pair_schedule_steps": (i32, [i64, i64, i64, i32, i32, P, P, P]),
            "qlora_pair_spans": (i32, [i64, i32, i32, i32, P, i32]),
            "qlora_launch_count": (ctypes.c_longlong, []),
            "qlora_set_kernel_events": (i32, [P, P]),
            "qlora_linear_fwd_noalloc": (i32, [P, i64, WP, P, P, i32, f32, P, P, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().qlora_status_string(int(code)).decode()


def _check(fn: str, rc: int):
    if rc != QLORA_OK:
        raise QLoRAError(fn, rc)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    # the raw handle of the current stream, without the Stream object around it (3.4 -> 0.3 us a call)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _on(stream, make):
    """make(), whose memory comes from the pool of the stream that the call runs on: a block that was freed on the
    current stream may still be in use by work queued there.  The current stream, where the caller reads the result,
    holds it as well."""
    if stream is None:
        return make()
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        out = make()
    for t in (out,) if isinstance(out, torch.Tensor) else (out.packed, out.codes, out.scale, out.mean):
        t.record_stream(here)
    return out


def _empty(shape: tuple, device, stream) -> torch.Tensor:
    return _on(stream, lambda: torch.empty(shape, dtype=torch.bfloat16, device=device))


def _bits(t: torch.Tensor) -> torch.Tensor:
    assert t.dtype == torch.bfloat16, t.dtype
    assert t.is_contiguous()
    return t


# --------------------------------------------------------------------------
@dataclass
class NF4Weight:
    """A quantized frozen weight: device tensors plus its logical shape."""
    packed: torch.Tensor   # uint8 [N, K/2]
    codes: torch.Tensor    # int8 [N*K/64]
    scale: torch.Tensor    # fp32 [G]
    mean: torch.Tensor     # fp32 [G]
    N: int
    K: int
    quant_type: int = QLORA_QUANT_NF4

    def c_struct(self) -> _Weight:
        return _Weight(self.packed.data_ptr(), self.codes.data_ptr(), self.scale.data_ptr(),
                       self.mean.data_ptr(), self.N, self.K, self.quant_type)

    @staticmethod
    def empty(N: int, K: int, device="cuda", quant_type: int = QLORA_QUANT_NF4) -> "NF4Weight":
        pb, nb, ng = nf4dq_sizes(N, K)
        return NF4Weight(torch.empty((N, K // 2), dtype=torch.uint8, device=device),
                         torch.empty(nb, dtype=torch.int8, device=device),
                         torch.empty(ng, dtype=torch.float32, device=device),
                         torch.empty(ng, dtype=torch.float32, device=device), N, K, quant_type)


def nf4_codebook() -> list:
    out = (ctypes.c_float * 16)()
    _check("nf4_codebook", lib().nf4_codebook(out))
    return list(out)


def quant4_codebook(quant_type: int) -> list:
    out = (ctypes.c_float * 16)()
    _check("quant4_codebook", lib().quant4_codebook(int(quant_type), out))
    return list(out)


def nf4dq_sizes(N: int, K: int):
    pb, nb, ng = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check("nf4dq_sizes", lib().nf4dq_sizes(N, K, ctypes.byref(pb), ctypes.byref(nb), ctypes.byref(ng)))
    return pb.value, nb.value, ng.value


def nf4_quantize_dq(W: torch.Tensor, out: NF4Weight | None = None, stream=None) -> NF4Weight:
    """bf16 W [N, K] (device) -> NF4Weight."""
    W = _bits(W)
    N, K = W.shape
    if out is None:
        out = _on(stream, lambda: NF4Weight.empty(N, K, W.device))
    _check("nf4_quantize_dq", lib().nf4_quantize_dq(_ptr(W), N, K, _ptr(out.packed), _ptr(out.codes),
                                                    _ptr(out.scale), _ptr(out.mean), _stream(stream)))
    return out


def quant4_quantize_dq(W: torch.Tensor, quant_type: int, out: NF4Weight | None = None, stream=None) -> NF4Weight:
    """bf16 W [N, K] (device) -> NF4Weight of the given quant type (NF4 or FP4)."""
    W = _bits(W)
    N, K = W.shape
    if out is None:
        out = _on(stream, lambda: NF4Weight.empty(N, K, W.device, quant_type))
    out.quant_type = int(quant_type)
    _check("quant4_quantize_dq", lib().quant4_quantize_dq(_ptr(W), N, K, int(quant_type), _ptr(out.packed),
                                                          _ptr(out.codes), _ptr(out.scale), _ptr(out.mean),
                                                          _stream(stream)))
    return out


def nf4_dequant_merge(w: NF4Weight, A, B, scaling: float, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Dense bf16 W' + scaling * B A (the merged weight of the adapted layer)."""
    if out is None:
        out = _empty((w.N, w.K), w.packed.device, stream)
    st = w.c_struct()
    _check("nf4_dequant_merge", lib().nf4_dequant_merge(ctypes.byref(st), _ptr(_bits(A)), _ptr(_bits(B)),
                                                        A.shape[0], float(scaling), _ptr(out), _stream(stream)))
    return out


QLORA_ADAM_BLOCK = 256


@dataclass
class AdamW8State:
    """8-bit moment states of n parameters (E4M3 codes + one fp32 scale per 256)."""
    m_code: torch.Tensor   # uint8 [n]
    m_scale: torch.Tensor  # fp32 [ceil(n / 256)]
    v_code: torch.Tensor   # uint8 [n]
    v_scale: torch.Tensor  # fp32 [ceil(n / 256)]

    @staticmethod
    def zeros(n: int, device="cuda") -> "AdamW8State":
        nb = (n + QLORA_ADAM_BLOCK - 1) // QLORA_ADAM_BLOCK
        return AdamW8State(torch.zeros(n, dtype=torch.uint8, device=device),
                           torch.zeros(nb, dtype=torch.float32, device=device),
                           torch.zeros(n, dtype=torch.uint8, device=device),
                           torch.zeros(nb, dtype=torch.float32, device=device))


def adamw_8bit_step(p: torch.Tensor, g: torch.Tensor, state: AdamW8State, step: int, lr: float,
                    beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                    stream=None) -> None:
    """In-place AdamW step of the bf16 parameters p with gradient g and 8-bit states."""
    p, g = _bits(p), _bits(g)
    _check("adamw_8bit_step", lib().adamw_8bit_step(
        _ptr(p), _ptr(g), p.numel(), _ptr(state.m_code), _ptr(state.m_scale), _ptr(state.v_code),
        _ptr(state.v_scale), int(step), float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
        _stream(stream)))


def nf4_dequant(w: NF4Weight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if out is None:
        out = _empty((w.N, w.K), w.packed.device, stream)
    st = w.c_struct()
    _check("nf4_dequant", lib().nf4_dequant(ctypes.byref(st), _ptr(out), _stream(stream)))
    return out


def qlora_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return int(lib().qlora_workspace_bytes(M, N, K, r))


def workspace(M: int, N: int, K: int, r: int, device="cuda") -> torch.Tensor:
    n = qlora_workspace_bytes(M, N, K, r)
    if n == 0:
        raise QLoRAError("qlora_workspace_bytes", -2)
    return torch.empty(n, dtype=torch.uint8, device=device)


def qlora_linear_fwd(X, w: NF4Weight, A, B, scaling: float, Y=None, T_out=None, ws=None, stream=None):
    """Y = X W'^T + s (X A^T) B^T; returns Y (and fills T_out when given)."""
    M = X.shape[0]
    if Y is None:
        Y = _empty((M, w.N), X.device, stream)
    if ws is None:
        ws = _on(stream, lambda: workspace(M, w.N, w.K, A.shape[0], X.device))
    st = w.c_struct()
    _check("qlora_linear_fwd", lib().qlora_linear_fwd(
        _ptr(_bits(X)), M, ctypes.byref(st), _ptr(_bits(A)), _ptr(_bits(B)), A.shape[0], float(scaling),
        _ptr(Y), _ptr(T_out), _ptr(ws), ws.numel(), _stream(stream)))
    return Y


def qlora_linear_bwd(X, dY, w: NF4Weight, A, B, scaling: float, T=None, dX=None, dA=None, dB=None, ws=None,
                     stream=None):
    """Returns (dX, dA, dB); the frozen weight gets no gradient."""
    M = X.shape[0]
    r = A.shape[0]
    dev = X.device
    if dX is None:
        dX = _empty((M, w.K), dev, stream)
    if dA is None:
        dA = _empty((r, w.K), dev, stream)
    if dB is None:
        dB = _empty((w.N, r), dev, stream)
    if ws is None:
        ws = _on(stream, lambda: workspace(M, w.N, w.K, r, dev))
    st = w.c_struct()
    _check("qlora_linear_bwd", lib().qlora_linear_bwd(
        _ptr(_bits(X)), _ptr(_bits(dY)), M, ctypes.byref(st), _ptr(_bits(A)), _ptr(_bits(B)), r, float(scaling),
        _ptr(T), _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(), _stream(stream)))
    return dX, dA, dB


def qlora_dropout_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return int(lib().qlora_dropout_workspace_bytes(M, N, K, r))


def dropout_workspace(M: int, N: int, K: int, r: int, device="cuda") -> torch.Tensor:
    n = qlora_dropout_workspace_bytes(M, N, K, r)
    if n == 0:
        raise QLoRAError("qlora_dropout_workspace_bytes", -2)
    return torch.empty(n, dtype=torch.uint8, device=device)


def qlora_linear_fwd_dropout(X, w: NF4Weight, A, B, scaling: float, dropout_p: float, seed: int, offset: int,
                             Y=None, T_out=None, ws=None, stream=None):
    """qlora_linear_fwd with LoRA dropout on the branch input (mask from (seed, offset))."""
    M = X.shape[0]
    if Y is None:
        Y = _empty((M, w.N), X.device, stream)
    if ws is None:
        ws = _on(stream, lambda: dropout_workspace(M, w.N, w.K, A.shape[0], X.device))
    st = w.c_struct()
    _check("qlora_linear_fwd_dropout", lib().qlora_linear_fwd_dropout(
        _ptr(_bits(X)), M, ctypes.byref(st), _ptr(_bits(A)), _ptr(_bits(B)), A.shape[0], float(scaling),
        float(dropout_p), int(seed), int(offset), _ptr(Y), _ptr(T_out), _ptr(ws), ws.numel(), _stream(stream)))
    return Y


def qlora_linear_bwd_dropout(X, dY, w: NF4Weight, A, B, scaling: float, dropout_p: float, seed: int, offset: int,
                             T=None, dX=None, dA=None, dB=None, ws=None, stream=None):
    """qlora_linear_bwd under the same LoRA dropout mask as the forward; returns (dX, dA, dB)."""
    M = X.shape[0]
    r = A.shape[0]
    dev = X.device
    if dX is None:
        dX = _empty((M, w.K), dev, stream)
    if dA is None:
        dA = _empty((r, w.K), dev, stream)
    if dB is None:
        dB = _empty((w.N, r), dev, stream)
    if ws is None:
        ws = _on(stream, lambda: dropout_workspace(M, w.N, w.K, r, dev))
    st = w.c_struct()
    _check("qlora_linear_bwd_dropout", lib().qlora_linear_bwd_dropout(
        _ptr(_bits(X)), _ptr(_bits(dY)), M, ctypes.byref(st), _ptr(_bits(A)), _ptr(_bits(B)), r, float(scaling),
        float(dropout_p), int(seed), int(offset), _ptr(T), _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(),
        _stream(stream)))
    return dX, dA, dB


# --------------------------------------------------------------------------
# 8-bit activation checkpoints
# --------------------------------------------------------------------------
def _need(t, name: str, dtype, shape: tuple) -> int:
    """The address of t, a dense tensor of this type and shape on the current device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape:
        got = f"{t.dtype} {tuple(t.shape)}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: {dtype} {shape} wanted, got {got}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    _on_device(t, name)
    return t.data_ptr()


def _on_device(t, name: str):
    if not t.is_cuda or t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: on {t.device}, not on the current CUDA device")


def _rows(t, name: str):
    """t is a [M, V] tensor of logits or their gradient, whose rows are dense."""
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.bfloat16, torch.float32) or t.dim() != 2:
        got = f"{t.dtype} {tuple(t.shape)}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: bf16 or fp32 [M, V] wanted, got {got}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row are not adjacent")
    _on_device(t, name)


_step_mod = None


def _step():
    """The extension that marshals the calls below (raises if it has not been built)."""
    global _step_mod
    if _step_mod is None:
        lib()
        from . import _step as mod
        mod.bind(QLoRAError, _need, _rows)
        _step_mod = mod
    return _step_mod


def _run(stream, fn, *args, ws=None):
    """fn(*args, stream handle); the outputs.

    On a stream that is not the current one, what fn allocates comes from that stream's pool: a block that was freed
    on the current stream may still be in use by work queued there.  Outputs go back to a pool only when the work
    queued by then on both streams is done (the current one is where the caller reads them)."""
    if stream is None:
        return fn(*args, None)
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        out = fn(*args, stream.cuda_stream)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(stream)
            t.record_stream(here)
    if ws is not None:
        ws.record_stream(stream)
    return out


@dataclass
class Act8Tensor:
    """An activation [M, K] kept in 8 bits: codes and one scale byte per 32 values of a row."""
    codes: torch.Tensor    # uint8 [M, K]
    scales: torch.Tensor   # uint8 [M, K / 32]
    M: int
    K: int
    fmt: int = QLORA_ACT8_INT8

    def c_struct(self) -> _Act8:
        return _Act8(_need(self.codes, "codes", torch.uint8, (self.M, self.K)),
                     _need(self.scales, "scales", torch.uint8, (self.M, self.K // QLORA_ACT8_BLOCK)), self.M, self.K,
                     self.fmt)

    @staticmethod
    def empty(M: int, K: int, device="cuda", fmt: int = QLORA_ACT8_INT8) -> "Act8Tensor":
        act8_sizes(M, K)
        return Act8Tensor(torch.empty((M, K), dtype=torch.uint8, device=device),
                          torch.empty((M, K // QLORA_ACT8_BLOCK), dtype=torch.uint8, device=device), M, K, fmt)


def act8_sizes(M: int, K: int):
    """(bytes of the codes, bytes of the scales) of an [M, K] checkpoint."""
    cb, sb = ctypes.c_int64(), ctypes.c_int64()
    _check("act8_sizes", lib().act8_sizes(M, K, ctypes.byref(cb), ctypes.byref(sb)))
    return cb.value, sb.value


def act8_quantize(X: torch.Tensor, fmt: int = QLORA_ACT8_INT8, out: Act8Tensor | None = None,
                  stream=None) -> Act8Tensor:
    """bf16 X [M, K] (device) -> 8-bit checkpoint."""
    if out is None:
        codes, scales = _run(stream, _step().act8_quantize, X, fmt, None, None)
        return Act8Tensor(codes, scales, *X.shape, int(fmt))
    if (out.M, out.K) != X.shape:
        raise ValueError(f"out: a checkpoint of {tuple(X.shape)} wanted, got {(out.M, out.K)}")
    _run(stream, _step().act8_quantize, X, fmt, out.codes, out.scales)
    out.fmt = int(fmt)
    return out


def act8_dequant(x: Act8Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """8-bit checkpoint -> the bf16 tensor it stands for."""
    return _run(stream, _step().act8_dequant, x.codes, x.scales, x.M, x.K, x.fmt, out)


def qlora_act8_workspace_bytes(M: int, N: int, K: int, r: int, dropout: bool = False) -> int:
    return int(lib().qlora_act8_workspace_bytes(M, N, K, r, int(dropout)))


def act8_workspace(M: int, N: int, K: int, r: int, dropout: bool = False, device="cuda") -> torch.Tensor:
    n = qlora_act8_workspace_bytes(M, N, K, r, dropout)
    if n == 0:
        raise QLoRAError("qlora_act8_workspace_bytes", -2)
    return torch.empty(n, dtype=torch.uint8, device=device)


def qlora_linear_bwd_act8(X: Act8Tensor, dY, w: NF4Weight, A, B, scaling: float, T=None, dX=None, dA=None, dB=None,
                          dropout_p: float = 0.0, seed: int = 0, offset: int = 0, ws=None, stream=None):
    """qlora_linear_bwd (dropout_p > 0: qlora_linear_bwd_dropout) from an 8-bit checkpoint of X; (dX, dA, dB)."""
    return _run(stream, _step().qlora_linear_bwd_act8, X.codes, X.scales, X.M, X.K, X.fmt, w.packed, w.codes, w.scale,
                w.mean, w.N, w.K, w.quant_type, dY, A, B, scaling, dropout_p, seed, offset, T, dX, dA, dB, ws, ws=ws)


# --------------------------------------------------------------------------
# losses on logits
# --------------------------------------------------------------------------
def loss_workspace_bytes(M: int) -> int:
    return int(lib().loss_workspace_bytes(M))


def loss_workspace(M: int, device="cuda") -> torch.Tensor:
    n = loss_workspace_bytes(M)
    if n == 0:
        raise QLoRAError("loss_workspace_bytes", -2)
    return torch.empty(n, dtype=torch.uint8, device=device)


def token_logprob(logits: torch.Tensor, targets: torch.Tensor, logit_scale: float = 1.0, out=None,
                  stream=None) -> torch.Tensor:
    """fp32 [M]: log-probability of each row's target (0 where the target is outside [0, V))."""
    return _run(stream, _step().token_logprob, logits, targets, logit_scale, out)


@dataclass
class PreferenceOut:
    loss: torch.Tensor      # fp32 scalar
    rewards: torch.Tensor   # fp32 [2 P]
    logp: torch.Tensor      # fp32 [M]
    dlogits: torch.Tensor | None


def preference_loss(logits, targets, cu_seqlens, ref_logp, beta: float, kind: int = QLORA_PREF_SIGMOID,
                    label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                    logit_scale: float = 1.0, grad_scale: float = 1.0, dlogits=None, want_grad: bool = True, ws=None,
                    stream=None) -> PreferenceOut:
    """Paired preference loss over packed sequences, with the gradient of the logits.

    cu_seqlens int32 [2 P + 1]: pair p prefers sequence 2p to sequence 2p + 1.  ref_logp fp32 [M] or None.
    dlogits may be the logits themselves; with want_grad=False and no dlogits, the loss alone."""
    return PreferenceOut(*_run(stream, _step().preference_loss, logits, targets, cu_seqlens, ref_logp, beta, kind,
                               label_smoothing, margin, average, logit_scale, grad_scale, dlogits, want_grad, ws,
                               ws=ws))


@dataclass
class PolicyOut:
    stats: torch.Tensor     # fp32 [4]: loss, policy term, KL, weight of the clipped rows
    logp: torch.Tensor      # fp32 [M]
    dlogits: torch.Tensor | None


def policy_loss(logits, targets, advantages, weights, old_logp, ref_logp, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, logit_scale: float = 1.0, grad_scale: float = 1.0,
                dlogits=None, want_grad: bool = True, ws=None, stream=None) -> PolicyOut:
    """Clipped policy loss with a KL term, with the gradient of the logits.

    advantages, weights fp32 [M]; old_logp, ref_logp fp32 [M] or None (ratio 1, no KL term).
    dlogits may be the logits themselves; with want_grad=False and no dlogits, the loss alone."""
    return PolicyOut(*_run(stream, _step().policy_loss, logits, targets, advantages, weights, old_logp, ref_logp,
                           clip_low, clip_high, kl_coef, logit_scale, grad_scale, dlogits, want_grad, ws, ws=ws))


def qlora_device_status(reset: bool = True) -> int:
    return int(lib().qlora_device_status(1 if reset else 0))


def qlora_last_path() -> int:
    return int(lib().qlora_last_path())


def qlora_launch_count() -> int:
    return int(lib().qlora_launch_count())


def qlora_set_kernel_events(before, after) -> None:
    """Record torch.cuda.Event `before`/`after` around the next fused dequant-GEMM launch on this thread."""
    b = ctypes.c_void_p(before.cuda_event) if before is not None else None
    a = ctypes.c_void_p(after.cuda_event) if after is not None else None
    _check("qlora_set_kernel_events", lib().qlora_set_kernel_events(b, a))


def qlora_linear_fwd_noalloc(X, w: NF4Weight, A, B, scaling: float, Y=None, T_out=None, stream=None):
    """qlora_linear_fwd on the library's fixed static scratch (no workspace argument)."""
    M = X.shape[0]
    if Y is None:
        Y = _empty((M, w.N), X.device, stream)
    st = w.c_struct()
    _check("qlora_linear_fwd_noalloc", lib().qlora_linear_fwd_noalloc(
        _ptr(_bits(X)), M, ctypes.byref(st), _ptr(_bits(A)), _ptr(_bits(B)), A.shape[0], float(scaling),
        _ptr(Y), _ptr(T_out), _stream(stream)))
    return Y


def pair_schedule(M: int, n_out: int, pairs: int, bwd: bool, nsteps: int = 0):
    """(token tiles per weight stage, tile count, stream-K) of the SM-pair kernel; nsteps: reduction steps of 64, 0 for
    as many as give every pair a unit."""
    mt, nt, sk = ctypes.c_int(0), ctypes.c_int64(0), ctypes.c_int(0)
    _check("qlora_pair_schedule_steps", lib().qlora_pair_schedule_steps(
        M, n_out, nsteps, pairs, int(bwd), ctypes.byref(mt), ctypes.byref(nt), ctypes.byref(sk)))
    return mt.value, nt.value, bool(sk.value)


def pair_spans(ntiles: int, nsteps: int, pair: int, npairs: int):
    """The stream-K spans [(tile, first step, end step), ...] of one pair, in the order it takes them."""
    buf = (ctypes.c_int64 * 3 * 64)()
    n = lib().qlora_pair_spans(ntiles, nsteps, pair, npairs, buf, 64)
    if n < 0:
        _check("qlora_pair_spans", n)
    assert n <= 64
    return [(buf[i][0], buf[i][1], buf[i][2]) for i in range(n)]
