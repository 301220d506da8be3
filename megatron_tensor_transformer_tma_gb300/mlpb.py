"""ctypes binding of libmlpb (the C ABI declared in include/mlpb.h).

Argument marshalling only: torch tensors are checked for dtype, shape, device and
contiguity and passed as raw device pointers with the current CUDA stream.  Every
step of the computation runs in the library's CUDA kernels; there is no fallback.
Loading fails loudly when libmlpb.so has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import functools
import os

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libmlpb.so")

MLPB_OK = 0
MLPB_EINVAL = -1
MLPB_EUNSUPPORTED = -2
MLPB_ECUDA = -3
MLPB_ETIMEOUT = -4
MLPB_ENOMEM = -5

MLPB_ACT_GELU_TANH = 0
MLPB_ACT_SWIGLU = 1
MLPB_FLAG_FAULT_INJECT = 0x1
MLPB_FLAG_ACCUMULATE_GRADS = 0x2
MLPB_FLAG_RECOMPUTE_ACT = 0x4
MLPB_FLAG_FP8 = 0x8
MLPB_FLAG_BF16_OUT = 0x10
MLPB_FLAG_EMULATE_COPIES = 0x20
MLPB_FLAG_CHECKPOINT8 = 0x100

MLPB_NORM_NONE = 0
MLPB_NORM_LAYER = 1
MLPB_NORM_RMS = 2
MLPB_JOIN_STREAM_F32 = 0x1
MLPB_JOIN_BLOCK_F32 = 0x2
MLPB_JOIN_ACCUMULATE_GRADS = 0x4
MLPB_MOE_FAULT_INJECT = 0x2
MLPB_LINEAR8_OUT_F32 = 0x1
MLPB_LINEAR8_FAULT_INJECT = 0x2
MLPB_MUON_FAULT_INJECT = 0x1
ACT8_BLOCK = 32  # features that share a scale byte of an 8-bit activation checkpoint

# Every symbol include/mlpb.h declares.
EXPORTED = (
    "mlpb_create", "mlpb_destroy", "mlpb_workspace_size", "mlpb_saved_size", "mlpb_forward",
    "mlpb_backward", "mlpb_layernorm_sp_fwd", "mlpb_layernorm_sp_bwd", "mlpb_last_device_error",
    "mlpb_enable_timing", "mlpb_read_timings", "mlpb_status_str", "mlpb_bias_grad_noalloc",
    "mlpb_branch_forward", "mlpb_branch_backward", "mlpb_quantize_e4m3",
    "mlpb_act8_scales", "mlpb_act8_save", "mlpb_act8_grad",
    "mlpb_join_workspace_size", "mlpb_join_fwd", "mlpb_join_bwd",
    "mlpb_moe_create", "mlpb_moe_destroy", "mlpb_moe_workspace_size", "mlpb_moe_forward",
    "mlpb_moe_last_device_error",
    "mlpb_b128_sizes", "mlpb_b128_quantize",
    "mlpb_linear8_create", "mlpb_linear8_destroy", "mlpb_linear8_workspace_size",
    "mlpb_linear8_forward", "mlpb_linear8_backward", "mlpb_linear8_last_device_error",
    "mlpb_muon_create", "mlpb_muon_destroy", "mlpb_muon_workspace_size",
    "mlpb_muon_orthogonalize", "mlpb_muon_step", "mlpb_muon_last_device_error",
)


class mlpb_config(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("ffn", ctypes.c_int64),
        ("tp", ctypes.c_int32), ("act", ctypes.c_int32), ("has_bias", ctypes.c_int32),
        ("seq_parallel_ln", ctypes.c_int32), ("ln_eps", ctypes.c_float), ("flags", ctypes.c_uint32),
    ]


class mlpb_join_config(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("gate_groups", ctypes.c_int64),
        ("has_block", ctypes.c_int32), ("post_norm", ctypes.c_int32),
        ("pre_norm", ctypes.c_int32), ("eps", ctypes.c_float), ("flags", ctypes.c_uint32),
    ]


class mlpb_moe_config(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("max_tokens", "hidden", "ffn", "experts", "topk",
                                              "act", "normalize")] + [("flags", ctypes.c_uint32)]


class mlpb_linear8_config(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_int64), ("inputs", ctypes.c_int64),
                ("outputs", ctypes.c_int64), ("flags", ctypes.c_uint32)]


class mlpb_muon_config(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("steps", ctypes.c_int32), ("nesterov", ctypes.c_int32),
                ("coef", ctypes.c_float * 3), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("scale", ctypes.c_float),
                ("flags", ctypes.c_uint32)]


class mlpb_kernel_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("ms", ctypes.c_float), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double), ("kernels", ctypes.c_int32)]


class MLPBError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} ({status})")


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libmlpb.so and declares its signatures (idempotent)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                           "(the MLP block has no non-CUDA implementation)")
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    I32, I64 = ctypes.c_int32, ctypes.c_int64
    H = ctypes.c_void_p
    sig = {
        "mlpb_create": (I, [ctypes.POINTER(mlpb_config), ctypes.POINTER(H)]),
        "mlpb_destroy": (None, [H]),
        "mlpb_workspace_size": (I, [H, ctypes.POINTER(Z)]),
        "mlpb_saved_size": (I, [H, ctypes.POINTER(Z), ctypes.POINTER(Z)]),
        "mlpb_forward": (I, [H, P, P, P, P, P, P, P, P, P, P]),
        "mlpb_backward": (I, [H, P, P, P, P, P, P, P, P, P, P, P, P, P]),
        "mlpb_layernorm_sp_fwd": (I, [H, P, P, P, P, P, P, P]),
        "mlpb_layernorm_sp_bwd": (I, [H, P, P, P, P, P, P, P, P, P, P]),
        "mlpb_last_device_error": (I, [H, P]),
        "mlpb_enable_timing": (I, [H, I]),
        "mlpb_read_timings": (I, [H, ctypes.POINTER(mlpb_kernel_time), I, ctypes.POINTER(I)]),
        "mlpb_status_str": (ctypes.c_char_p, [I]),
        "mlpb_bias_grad_noalloc": (I, [P, ctypes.c_int64, ctypes.c_int64, P, P]),
        "mlpb_branch_forward": (I, [H] + [P] * 15),
        "mlpb_branch_backward": (I, [H] + [P] * 19),
        "mlpb_quantize_e4m3": (I, [P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, P, P, P, P,
                                   P]),
        "mlpb_act8_scales": (I, [I32, I64, I32, ctypes.POINTER(I64)]),
        "mlpb_act8_save": (I, [I32, I64, I64, I32] + [P] * 5),
        "mlpb_act8_grad": (I, [I32, I64, I64, I32] + [P] * 6),
        "mlpb_join_workspace_size": (I, [ctypes.POINTER(mlpb_join_config), ctypes.POINTER(Z)]),
        "mlpb_join_fwd": (I, [ctypes.POINTER(mlpb_join_config)] + [P] * 12),
        "mlpb_join_bwd": (I, [ctypes.POINTER(mlpb_join_config)] + [P] * 21),
        "mlpb_moe_create": (I, [ctypes.POINTER(mlpb_moe_config), ctypes.POINTER(H)]),
        "mlpb_moe_destroy": (None, [H]),
        "mlpb_moe_workspace_size": (I, [H, ctypes.POINTER(Z)]),
        "mlpb_moe_forward": (I, [H, I64] + [P] * 9),
        "mlpb_moe_last_device_error": (I, [H, P]),
        "mlpb_b128_sizes": (I, [I64, I64, ctypes.POINTER(I64), ctypes.POINTER(Z)]),
        "mlpb_b128_quantize": (I, [P, I32, I64, I64, I32] + [P] * 5),
        "mlpb_linear8_create": (I, [ctypes.POINTER(mlpb_linear8_config), ctypes.POINTER(H)]),
        "mlpb_linear8_destroy": (None, [H]),
        "mlpb_linear8_workspace_size": (I, [H, ctypes.POINTER(Z)]),
        "mlpb_linear8_forward": (I, [H, I64] + [P] * 8),
        "mlpb_linear8_backward": (I, [H, I64] + [P] * 7 + [I32, P, P]),
        "mlpb_linear8_last_device_error": (I, [H, P]),
        "mlpb_muon_create": (I, [ctypes.POINTER(mlpb_muon_config), ctypes.POINTER(H)]),
        "mlpb_muon_destroy": (None, [H]),
        "mlpb_muon_workspace_size": (I, [H, ctypes.POINTER(Z)]),
        "mlpb_muon_orthogonalize": (I, [H, P, I32, P, P, P]),
        "mlpb_muon_step": (I, [H] + [P] * 7),
        "mlpb_muon_last_device_error": (I, [H, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load_library().mlpb_status_str(status).decode()


def _check(status: int, where: str):
    if status != MLPB_OK:
        raise MLPBError(status, where)


def _ptr(t, dtype=None, shape=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _arg(t, dtype, shape, name, dev):
    """The data pointer of a contiguous CUDA tensor of this dtype and shape on CUDA device
    number `dev` (None passes)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    raise ValueError(f"{name}: on cuda:{t.get_device()}, other tensors on cuda:{dev}")


def _cuda_index(t, name):
    """The CUDA device number that a call's tensors live on, taken from its first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    return t.get_device()


# The current stream's handle without a Stream object around it, where torch offers that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on_device(dev, fn, args, stream):
    """The result of a library function for `args` and a stream (None: the current one of device
    `dev`), with that device current: the library works on the current device."""
    if stream is None:
        s = _raw_stream(dev)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if dev == torch.cuda.current_device():
        return fn(*args, s)
    with torch.cuda.device(dev):
        return fn(*args, s)


def _call_on(dev, name, args, stream):
    """The same by the function's name, raising for a status that is not MLPB_OK."""
    _check(_on_device(dev, getattr(load_library(), name), args, stream), name)


def _on(stream, device):
    """A context in which new tensors on `device` belong to the stream that the call will run on."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _new(shape, dtype, device, stream):
    """A new tensor that belongs to the stream that the call will run on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _device(device):
    """The torch.device of a plan; "cuda" is the device that is current now, for good."""
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:
        d = torch.device("cuda", torch.cuda.current_device())
    return d


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


@dataclasses.dataclass
class Handle:
    ptr: int
    cfg: mlpb_config

    @property
    def shape(self):
        c = self.cfg
        return c.tokens, c.hidden, c.ffn, c.tp


def make_config(tokens, hidden, ffn, tp, act="gelu", has_bias=True, seq_parallel_ln=False,
                ln_eps=1e-5, flags=0) -> mlpb_config:
    return mlpb_config(tokens, hidden, ffn, tp,
                       MLPB_ACT_SWIGLU if act == "swiglu" else MLPB_ACT_GELU_TANH,
                       1 if has_bias else 0, 1 if seq_parallel_ln else 0, ln_eps, flags)


def mlpb_create(cfg: mlpb_config) -> Handle:
    h = ctypes.c_void_p()
    _check(load_library().mlpb_create(ctypes.byref(cfg), ctypes.byref(h)), "mlpb_create")
    return Handle(h.value, cfg)


def mlpb_destroy(h: Handle):
    if h is not None and h.ptr:
        load_library().mlpb_destroy(h.ptr)
        h.ptr = 0


def mlpb_workspace_size(h: Handle) -> int:
    n = ctypes.c_size_t()
    _check(load_library().mlpb_workspace_size(h.ptr, ctypes.byref(n)), "mlpb_workspace_size")
    return n.value


def mlpb_saved_size(h: Handle):
    z, a = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().mlpb_saved_size(h.ptr, ctypes.byref(z), ctypes.byref(a)),
           "mlpb_saved_size")
    return z.value, a.value


def out_dtype(c):
    """dtype of Y, dX (and the LayerNorm backward's dXn): bf16 under MLPB_FLAG_BF16_OUT."""
    return torch.bfloat16 if c.flags & MLPB_FLAG_BF16_OUT else torch.float32


def _w1_shape(c):
    fs = c.ffn // c.tp
    return (c.tp, 2, fs, c.hidden) if c.act == MLPB_ACT_SWIGLU else (c.tp, fs, c.hidden)


def _saved_z(h: Handle):
    """(dtype, shape) of Zsaved: bf16 [T][F1], or the bytes of an 8-bit checkpoint."""
    c = h.cfg
    f1 = 2 * c.ffn if c.act == MLPB_ACT_SWIGLU else c.ffn
    if c.flags & MLPB_FLAG_CHECKPOINT8:
        return torch.uint8, (c.tokens * f1 + c.tokens * f1 // ACT8_BLOCK,)
    return torch.bfloat16, (c.tokens, f1)


def mlpb_forward(h: Handle, X, W1, b1, W2, b2, Y, Zsaved, Asaved, workspace=None, stream=None):
    c = h.cfg
    T, Hd, F, t = c.tokens, c.hidden, c.ffn, c.tp
    bf = torch.bfloat16
    args = [
        _ptr(X, bf, (T, Hd), "X"), _ptr(W1, bf, _w1_shape(c), "W1"), _ptr(b1, bf, (F,), "b1"),
        _ptr(W2, bf, (t, Hd, F // t), "W2"), _ptr(b2, bf, (Hd,), "b2"),
        _ptr(Y, out_dtype(c), (T, Hd), "Y"), _ptr(Zsaved, *_saved_z(h), "Zsaved"),
        _ptr(Asaved, bf, (T, F), "Asaved"), _ptr(workspace, None, None, "workspace"),
    ]
    _check(load_library().mlpb_forward(h.ptr, *args, _stream(stream)), "mlpb_forward")


def mlpb_backward(h: Handle, X, W1, W2, Zsaved, Asaved, dY, dX, dW1, dW2, db1, db2, workspace,
                  stream=None):
    c = h.cfg
    T, Hd, F, t = c.tokens, c.hidden, c.ffn, c.tp
    bf, f32 = torch.bfloat16, torch.float32
    args = [
        _ptr(X, bf, (T, Hd), "X"), _ptr(W1, bf, _w1_shape(c), "W1"),
        _ptr(W2, bf, (t, Hd, F // t), "W2"), _ptr(Zsaved, *_saved_z(h), "Zsaved"),
        _ptr(Asaved, bf, (T, F), "Asaved"), _ptr(dY, bf, (T, Hd), "dY"),
        _ptr(dX, out_dtype(c), (T, Hd), "dX"), _ptr(dW1, f32, _w1_shape(c), "dW1"),
        _ptr(dW2, f32, (t, Hd, F // t), "dW2"), _ptr(db1, f32, (F,), "db1"),
        _ptr(db2, f32, (Hd,), "db2"), _ptr(workspace, None, None, "workspace"),
    ]
    _check(load_library().mlpb_backward(h.ptr, *args, _stream(stream)), "mlpb_backward")


def mlpb_layernorm_sp_fwd(h: Handle, X, gamma, beta, Xn, mean, rstd, stream=None):
    c = h.cfg
    T, Hd = c.tokens, c.hidden
    bf, f32 = torch.bfloat16, torch.float32
    args = [_ptr(X, bf, (T, Hd), "X"), _ptr(gamma, bf, (Hd,), "gamma"),
            _ptr(beta, bf, (Hd,), "beta"), _ptr(Xn, bf, (T, Hd), "Xn"),
            _ptr(mean, f32, (T,), "mean"), _ptr(rstd, f32, (T,), "rstd")]
    _check(load_library().mlpb_layernorm_sp_fwd(h.ptr, *args, _stream(stream)),
           "mlpb_layernorm_sp_fwd")


def mlpb_layernorm_sp_bwd(h: Handle, X, gamma, mean, rstd, dXn, dX, dgamma, dbeta, workspace,
                          stream=None):
    c = h.cfg
    T, Hd = c.tokens, c.hidden
    bf, f32 = torch.bfloat16, torch.float32
    args = [_ptr(X, bf, (T, Hd), "X"), _ptr(gamma, bf, (Hd,), "gamma"),
            _ptr(mean, f32, (T,), "mean"), _ptr(rstd, f32, (T,), "rstd"),
            _ptr(dXn, out_dtype(c), (T, Hd), "dXn"), _ptr(dX, out_dtype(c), (T, Hd), "dX"),
            _ptr(dgamma, f32, (Hd,), "dgamma"), _ptr(dbeta, f32, (Hd,), "dbeta"),
            _ptr(workspace, None, None, "workspace")]
    _check(load_library().mlpb_layernorm_sp_bwd(h.ptr, *args, _stream(stream)),
           "mlpb_layernorm_sp_bwd")


def mlpb_branch_forward(h: Handle, X, gamma, beta, W1, b1, W2, b2, Y, Xn, mean, rstd, Zsaved,
                        Asaved, workspace=None, stream=None):
    c = h.cfg
    T, Hd, F, t = c.tokens, c.hidden, c.ffn, c.tp
    bf, f32 = torch.bfloat16, torch.float32
    args = [
        _ptr(X, bf, (T, Hd), "X"), _ptr(gamma, bf, (Hd,), "gamma"), _ptr(beta, bf, (Hd,), "beta"),
        _ptr(W1, bf, _w1_shape(c), "W1"), _ptr(b1, bf, (F,), "b1"),
        _ptr(W2, bf, (t, Hd, F // t), "W2"), _ptr(b2, bf, (Hd,), "b2"),
        _ptr(Y, out_dtype(c), (T, Hd), "Y"), _ptr(Xn, bf, (T, Hd), "Xn"),
        _ptr(mean, f32, (T,), "mean"),
        _ptr(rstd, f32, (T,), "rstd"), _ptr(Zsaved, *_saved_z(h), "Zsaved"),
        _ptr(Asaved, bf, (T, F), "Asaved"), _ptr(workspace, None, None, "workspace"),
    ]
    _check(load_library().mlpb_branch_forward(h.ptr, *args, _stream(stream)),
           "mlpb_branch_forward")


def mlpb_branch_backward(h: Handle, X, gamma, W1, W2, Xn, mean, rstd, Zsaved, Asaved, dY, dX,
                         dW1, dW2, db1, db2, dgamma, dbeta, workspace, stream=None):
    c = h.cfg
    T, Hd, F, t = c.tokens, c.hidden, c.ffn, c.tp
    bf, f32 = torch.bfloat16, torch.float32
    args = [
        _ptr(X, bf, (T, Hd), "X"), _ptr(gamma, bf, (Hd,), "gamma"),
        _ptr(W1, bf, _w1_shape(c), "W1"), _ptr(W2, bf, (t, Hd, F // t), "W2"),
        _ptr(Xn, bf, (T, Hd), "Xn"), _ptr(mean, f32, (T,), "mean"), _ptr(rstd, f32, (T,), "rstd"),
        _ptr(Zsaved, *_saved_z(h), "Zsaved"), _ptr(Asaved, bf, (T, F), "Asaved"),
        _ptr(dY, bf, (T, Hd), "dY"), _ptr(dX, out_dtype(c), (T, Hd), "dX"),
        _ptr(dW1, f32, _w1_shape(c), "dW1"), _ptr(dW2, f32, (t, Hd, F // t), "dW2"),
        _ptr(db1, f32, (F,), "db1"), _ptr(db2, f32, (Hd,), "db2"),
        _ptr(dgamma, f32, (Hd,), "dgamma"), _ptr(dbeta, f32, (Hd,), "dbeta"),
        _ptr(workspace, None, None, "workspace"),
    ]
    _check(load_library().mlpb_branch_backward(h.ptr, *args, _stream(stream)),
           "mlpb_branch_backward")


def mlpb_quantize_e4m3(inp, q=None, qt=None, amax=None, scale_exp=None, stream=None):
    """E4M3 codes (uint8 tensors) of a bf16 CUDA tensor [rows][cols] or [batches][rows][cols]
    with one power-of-two scale; q in the input's layout, qt with the last two dimensions
    swapped.  Returns (amax bits as an int32 CUDA tensor, scale exponent int32 CUDA tensor)."""
    shape = tuple(inp.shape)
    b, r, c = (1,) + shape if len(shape) == 2 else shape
    dev = inp.device
    if amax is None:
        amax = torch.empty(1, dtype=torch.int32, device=dev)
    if scale_exp is None:
        scale_exp = torch.empty(1, dtype=torch.int32, device=dev)
    args = [_ptr(inp, torch.bfloat16, None, "in"), b, r, c,
            _ptr(q, torch.uint8, shape, "q"),
            _ptr(qt, torch.uint8, shape[:-2] + (c, r), "qt"),
            _ptr(amax, torch.int32, (1,), "amax"), _ptr(scale_exp, torch.int32, (1,), "scale_exp")]
    _check(load_library().mlpb_quantize_e4m3(*args, _stream(stream)), "mlpb_quantize_e4m3")
    return amax, scale_exp


_ACTS = {"gelu": MLPB_ACT_GELU_TANH, "swiglu": MLPB_ACT_SWIGLU}


@functools.lru_cache(maxsize=None)
def mlpb_act8_scales(act, ffn, tp=1) -> int:
    """Scale bytes of a row of an 8-bit activation checkpoint (act: "gelu" or "swiglu")."""
    n = ctypes.c_int64()
    _check(load_library().mlpb_act8_scales(_ACTS[act], ffn, tp, ctypes.byref(n)),
           "mlpb_act8_scales")
    return n.value


def mlpb_act8_save(act, Z, A, codes, scales, tp=1, stream=None):
    """Saves fc1's bf16 output Z ([T][F], or [T][2F] as [T][tp][2][Fs] for "swiglu") as int8
    codes (Z's shape) and uint8 scales [T][mlpb_act8_scales()], and writes A = act(Z) [T][F]
    bf16 unless A is None."""
    dev = _cuda_index(Z, "Z")
    if Z.dim() != 2:
        raise ValueError(f"Z: expected [tokens][features], got {tuple(Z.shape)}")
    T, f1 = Z.shape
    F = f1 // 2 if act == "swiglu" else f1
    f1 = 2 * F if act == "swiglu" else F  # an odd width fails Z's shape check
    nb = mlpb_act8_scales(act, F, tp)
    args = [_ACTS[act], T, F, tp, _arg(Z, torch.bfloat16, (T, f1), "Z", dev),
            _arg(A, torch.bfloat16, (T, F), "A", dev),
            _arg(codes, torch.int8, (T, f1), "codes", dev),
            _arg(scales, torch.uint8, (T, nb), "scales", dev)]
    _call_on(dev, "mlpb_act8_save", args, stream)


def mlpb_act8_grad(act, dA, codes, scales, dZ, A=None, tp=1, stream=None):
    """dZ = dA act'(z) (bf16, codes' shape) for the values z that an 8-bit checkpoint stands
    for, and A = act(z) [T][F] bf16 unless A is None; dA [T][F] bf16."""
    dev = _cuda_index(dA, "dA")
    if dA.dim() != 2:
        raise ValueError(f"dA: expected [tokens][features], got {tuple(dA.shape)}")
    T, F = dA.shape
    f1 = 2 * F if act == "swiglu" else F
    nb = mlpb_act8_scales(act, F, tp)
    args = [_ACTS[act], T, F, tp, _arg(dA, torch.bfloat16, (T, F), "dA", dev),
            _arg(codes, torch.int8, (T, f1), "codes", dev),
            _arg(scales, torch.uint8, (T, nb), "scales", dev),
            _arg(dZ, torch.bfloat16, (T, f1), "dZ", dev),
            _arg(A, torch.bfloat16, (T, F), "A", dev)]
    _call_on(dev, "mlpb_act8_grad", args, stream)


_NORMS = {"none": MLPB_NORM_NONE, "layer": MLPB_NORM_LAYER, "rms": MLPB_NORM_RMS}


def make_join_config(tokens, hidden, post_norm="none", pre_norm="none", gate_groups=0, eps=1e-5,
                     stream_dtype=torch.bfloat16, block_dtype=torch.bfloat16, accumulate=False,
                     has_block=True) -> mlpb_join_config:
    """Norms by name ("none", "layer", "rms"); dtypes torch.bfloat16 or torch.float32."""
    for t in (stream_dtype, block_dtype):
        if t not in (torch.bfloat16, torch.float32):
            raise TypeError(f"join: tensors are bfloat16 or float32, not {t}")
    flags = ((MLPB_JOIN_STREAM_F32 if stream_dtype == torch.float32 else 0)
             | (MLPB_JOIN_BLOCK_F32 if block_dtype == torch.float32 else 0)
             | (MLPB_JOIN_ACCUMULATE_GRADS if accumulate else 0))
    return mlpb_join_config(tokens, hidden, gate_groups, 1 if has_block else 0,
                            _NORMS[post_norm], _NORMS[pre_norm], eps, flags)


def _join_types(c):
    return (torch.float32 if c.flags & MLPB_JOIN_STREAM_F32 else torch.bfloat16,
            torch.float32 if c.flags & MLPB_JOIN_BLOCK_F32 else torch.bfloat16)


def mlpb_join_workspace_size(cfg: mlpb_join_config) -> int:
    """Bytes of mlpb_join_bwd's workspace on the current CUDA device."""
    n = ctypes.c_size_t()
    _check(load_library().mlpb_join_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "mlpb_join_workspace_size")
    return n.value


def mlpb_join_fwd(cfg, X, Y, res_scale, gate, gamma_post, beta_post, gamma_pre, beta_pre, Xout, Xn,
                  stats, stream=None):
    """The join between two blocks (include/mlpb.h): Xout = res_scale X + gate norm_post(Y),
    Xn = norm_pre(Xout), and the rows' statistics for the backward."""
    dev = _cuda_index(X, "X")
    T, H = cfg.tokens, cfg.hidden
    bf, f32 = torch.bfloat16, torch.float32
    xt, yt = _join_types(cfg)
    row, vec = (T, H), (H,)
    args = [ctypes.byref(cfg), _arg(X, xt, row, "X", dev), _arg(Y, yt, row, "Y", dev),
            _arg(res_scale, f32, (1,), "res_scale", dev),
            _arg(gate, bf, (cfg.gate_groups, H), "gate", dev),
            _arg(gamma_post, bf, vec, "gamma_post", dev),
            _arg(beta_post, bf, vec, "beta_post", dev),
            _arg(gamma_pre, bf, vec, "gamma_pre", dev), _arg(beta_pre, bf, vec, "beta_pre", dev),
            _arg(Xout, xt, row, "Xout", dev), _arg(Xn, bf, row, "Xn", dev),
            _arg(stats, f32, (T, 4), "stats", dev)]
    _call_on(dev, "mlpb_join_fwd", args, stream)


def mlpb_join_bwd(cfg, X, Y, Xout, stats, res_scale, gate, gamma_post, beta_post, gamma_pre, dXout,
                  dXn, dX, dY, dres_scale, dgate, dgamma_post, dbeta_post, dgamma_pre, dbeta_pre,
                  workspace, stream=None):
    """Backward of mlpb_join_fwd for the gradients dXout and dXn of its outputs."""
    dev = _cuda_index(dX, "dX")
    T, H = cfg.tokens, cfg.hidden
    bf, f32 = torch.bfloat16, torch.float32
    xt, yt = _join_types(cfg)
    row, vec, gates = (T, H), (H,), (cfg.gate_groups, H)
    if workspace is not None and workspace.nbytes < _join_ws_of(bytes(cfg), dev):
        raise ValueError("workspace: smaller than mlpb_join_workspace_size()")
    args = [ctypes.byref(cfg), _arg(X, xt, row, "X", dev), _arg(Y, yt, row, "Y", dev),
            _arg(Xout, xt, row, "Xout", dev), _arg(stats, f32, (T, 4), "stats", dev),
            _arg(res_scale, f32, (1,), "res_scale", dev), _arg(gate, bf, gates, "gate", dev),
            _arg(gamma_post, bf, vec, "gamma_post", dev),
            _arg(beta_post, bf, vec, "beta_post", dev),
            _arg(gamma_pre, bf, vec, "gamma_pre", dev), _arg(dXout, xt, row, "dXout", dev),
            _arg(dXn, yt, row, "dXn", dev), _arg(dX, xt, row, "dX", dev),
            _arg(dY, bf, row, "dY", dev), _arg(dres_scale, f32, (1,), "dres_scale", dev),
            _arg(dgate, f32, gates, "dgate", dev),
            _arg(dgamma_post, f32, vec, "dgamma_post", dev),
            _arg(dbeta_post, f32, vec, "dbeta_post", dev),
            _arg(dgamma_pre, f32, vec, "dgamma_pre", dev),
            _arg(dbeta_pre, f32, vec, "dbeta_pre", dev),
            _arg(workspace, torch.uint8, None if workspace is None else workspace.shape,
                 "workspace", dev)]
    _call_on(dev, "mlpb_join_bwd", args, stream)


def _join_ws(cfg, dev):
    return _join_ws_of(bytes(cfg), _device(dev).index)


@functools.lru_cache(maxsize=1024)
def _join_ws_of(cfg, dev):
    """A function of the configuration's bytes and the device's number of SMs alone."""
    with torch.cuda.device(dev):
        return mlpb_join_workspace_size(mlpb_join_config.from_buffer_copy(cfg))


@dataclasses.dataclass
class MoEHandle:
    ptr: int
    cfg: mlpb_moe_config
    device: int  # CUDA device number it was created on


def make_moe_config(max_tokens, hidden, ffn, experts, topk, act="swiglu", normalize=True,
                    flags=0) -> mlpb_moe_config:
    return mlpb_moe_config(max_tokens, hidden, ffn, experts, topk, _ACTS[act],
                           1 if normalize else 0, flags)


def mlpb_moe_create(cfg: mlpb_moe_config) -> MoEHandle:
    """A mixture-of-experts handle on the current CUDA device."""
    h = ctypes.c_void_p()
    _check(load_library().mlpb_moe_create(ctypes.byref(cfg), ctypes.byref(h)), "mlpb_moe_create")
    return MoEHandle(h.value, cfg, torch.cuda.current_device())


def mlpb_moe_destroy(h: MoEHandle):
    if h is not None and h.ptr:
        load_library().mlpb_moe_destroy(h.ptr)
        h.ptr = 0


def mlpb_moe_workspace_size(h: MoEHandle) -> int:
    n = ctypes.c_size_t()
    _check(load_library().mlpb_moe_workspace_size(h.ptr, ctypes.byref(n)),
           "mlpb_moe_workspace_size")
    return n.value


def mlpb_moe_forward(h: MoEHandle, X, Wr, W1, W2, Y, ids, weights, workspace, stream=None):
    """Router, experts and combination of the mixture-of-experts MLP for the rows of X
    (include/mlpb.h); ids int32 and weights fp32 [tokens][topk] receive the routing."""
    dev = _cuda_index(X, "X")
    if dev != h.device:
        raise ValueError(f"X: on cuda:{dev}, the handle on cuda:{h.device}")
    c = h.cfg
    if X.dim() != 2:
        raise ValueError(f"X: expected [tokens][hidden], got {tuple(X.shape)}")
    T, H, F, E = X.shape[0], c.hidden, c.ffn, c.experts
    bf = torch.bfloat16
    w1 = (E, 2, F, H) if c.act == MLPB_ACT_SWIGLU else (E, F, H)
    if workspace is not None and workspace.numel() * workspace.element_size() \
            < mlpb_moe_workspace_size(h):
        raise ValueError("workspace: smaller than mlpb_moe_workspace_size()")
    args = [h.ptr, T, _arg(X, bf, (T, H), "X", dev), _arg(Wr, bf, (E, H), "Wr", dev),
            _arg(W1, bf, w1, "W1", dev), _arg(W2, bf, (E, H, F), "W2", dev),
            _arg(Y, bf, (T, H), "Y", dev), _arg(ids, torch.int32, (T, c.topk), "ids", dev),
            _arg(weights, torch.float32, (T, c.topk), "weights", dev),
            _arg(workspace, torch.uint8, None if workspace is None else workspace.shape,
                 "workspace", dev)]
    _call_on(dev, "mlpb_moe_forward", args, stream)


def mlpb_moe_last_device_error(h: MoEHandle, stream=None) -> int:
    """The status code (MLPB_OK, MLPB_ETIMEOUT, MLPB_ECUDA) without raising, after the work of
    `stream` (None: the current one of the handle's device)."""
    return _on_device(h.device, load_library().mlpb_moe_last_device_error, [h.ptr], stream)


@functools.lru_cache(maxsize=4096)
def mlpb_b128_sizes(rows, cols):
    """(bytes of a row of codes, bytes of the scales) of a block-scaled E4M3 [rows][cols] matrix."""
    ld, n = ctypes.c_int64(), ctypes.c_size_t()
    _check(load_library().mlpb_b128_sizes(rows, cols, ctypes.byref(ld), ctypes.byref(n)),
           "mlpb_b128_sizes")
    return ld.value, n.value


def b128_empty(rows, cols, device):
    """Uninitialised codes [rows][ld] and scales of a [rows][cols] matrix (uint8)."""
    ld, n = mlpb_b128_sizes(rows, cols)
    return (torch.empty((rows, ld), dtype=torch.uint8, device=device),
            torch.empty(n, dtype=torch.uint8, device=device))


def _b128_args(q, rows, cols, name, dev):
    """Pointers of a (codes, scales) pair, or of None."""
    if q is None:
        return [None, None]
    ld, n = mlpb_b128_sizes(rows, cols)
    return [_arg(q[0], torch.uint8, (rows, ld), name + " codes", dev),
            _arg(q[1], torch.uint8, (n,), name + " scales", dev)]


def mlpb_b128_quantize(x, q=None, qt=None, square=False, stream=None):
    """Block-scaled E4M3 (include/mlpb.h) of a bf16 or fp32 matrix x [rows][cols] into q and/or of
    its transpose into qt, each a (codes, scales) pair of b128_empty()."""
    dev = _cuda_index(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x: expected [rows][cols], got {tuple(x.shape)}")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"x: expected bfloat16 or float32, got {x.dtype}")
    rows, cols = x.shape
    args = [_arg(x, x.dtype, x.shape, "x", dev), 1 if x.dtype == torch.float32 else 0, rows, cols,
            1 if square else 0, *_b128_args(q, rows, cols, "q", dev),
            *_b128_args(qt, cols, rows, "qt", dev)]
    _call_on(dev, "mlpb_b128_quantize", args, stream)


def b128_values(q, rows, cols):
    """What a (codes, scales) pair stands for, as fp64 [rows][cols] (torch operations: for tests
    and inspection; fp32's largest values are rounded to 2^128)."""
    codes, scales = q
    if rows == 0 or cols == 0:
        return torch.empty((rows, cols), dtype=torch.float64, device=codes.device)
    n = -(-cols // 128)
    tiles = -(-rows // 128)
    e = scales.view(-1, tiles, 32, 4, 4).permute(1, 3, 2, 0, 4).reshape(tiles * 128, -1)[:rows, :n]
    v = codes[:, :cols].contiguous().view(torch.float8_e4m3fn).double()
    e = e.to(torch.int32).repeat_interleave(128, 1)[:, :cols]
    return torch.where(e == 255, torch.full_like(v, float("nan")), v * torch.exp2(e.double() - 127))


@dataclasses.dataclass
class Linear8Handle:
    ptr: int
    cfg: mlpb_linear8_config
    device: int  # CUDA device number it was created on
    workspace_bytes: int


def mlpb_linear8_create(cfg: mlpb_linear8_config) -> Linear8Handle:
    """A linear layer's handle on the current CUDA device."""
    lib, h, n = load_library(), ctypes.c_void_p(), ctypes.c_size_t()
    _check(lib.mlpb_linear8_create(ctypes.byref(cfg), ctypes.byref(h)), "mlpb_linear8_create")
    _check(lib.mlpb_linear8_workspace_size(h.value, ctypes.byref(n)),
           "mlpb_linear8_workspace_size")
    return Linear8Handle(h.value, cfg, torch.cuda.current_device(), n.value)


def mlpb_linear8_destroy(h: Linear8Handle):
    if h is not None and h.ptr:
        load_library().mlpb_linear8_destroy(h.ptr)
        h.ptr = 0


def mlpb_linear8_workspace_size(h: Linear8Handle) -> int:
    return h.workspace_bytes


def _linear8_rows(h, t, cols, name):
    """(device, rows) of a call's first tensor [rows][cols]."""
    dev = _cuda_index(t, name)
    if dev != h.device:
        raise ValueError(f"{name}: on cuda:{dev}, the handle on cuda:{h.device}")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected [tokens][{cols}], got {tuple(t.shape)}")
    return dev, t.shape[0]


def _workspace(ws, need, dev):
    if ws is None:
        return None
    p = _arg(ws, torch.uint8, ws.shape, "workspace", dev)
    if ws.numel() < need:
        raise ValueError(f"workspace: {ws.numel()} bytes, {need} are needed")
    return p


def _linear8_out(c):
    return torch.float32 if c.flags & MLPB_LINEAR8_OUT_F32 else torch.bfloat16


def mlpb_linear8_forward(h, X, Wq, Y, Xt=None, workspace=None, stream=None):
    """Y = X W^T for the rows of X (include/mlpb.h); Wq, and Xt for the backward, are (codes,
    scales) pairs."""
    c = h.cfg
    K, N = c.inputs, c.outputs
    dev, T = _linear8_rows(h, X, K, "X")
    args = [h.ptr, T, _arg(X, torch.bfloat16, (T, K), "X", dev), *_b128_args(Wq, N, K, "Wq", dev),
            _arg(Y, _linear8_out(c), (T, N), "Y", dev), *_b128_args(Xt, K, T, "Xt", dev),
            _workspace(workspace, h.workspace_bytes, dev)]
    _call_on(dev, "mlpb_linear8_forward", args, stream)


def mlpb_linear8_backward(h, dY, Wt, Xt, dX, dW, accumulate=False, workspace=None, stream=None):
    """dX = dY W and dW (+)= dY^T X; either output may be None."""
    c = h.cfg
    K, N = c.inputs, c.outputs
    dev, T = _linear8_rows(h, dY, N, "dY")
    args = [h.ptr, T, _arg(dY, torch.bfloat16, (T, N), "dY", dev), *_b128_args(Wt, K, N, "Wt", dev),
            *_b128_args(Xt, K, T, "Xt", dev), _arg(dX, _linear8_out(c), (T, K), "dX", dev),
            _arg(dW, torch.float32, (N, K), "dW", dev), 1 if accumulate else 0,
            _workspace(workspace, h.workspace_bytes, dev)]
    _call_on(dev, "mlpb_linear8_backward", args, stream)


def mlpb_linear8_last_device_error(h: Linear8Handle, stream=None) -> int:
    """The status code (MLPB_OK, MLPB_ETIMEOUT, MLPB_ECUDA) without raising."""
    return _on_device(h.device, load_library().mlpb_linear8_last_device_error, [h.ptr], stream)


@dataclasses.dataclass
class MuonHandle:
    ptr: int
    cfg: mlpb_muon_config
    device: int  # CUDA device number it was created on
    workspace_bytes: int


def make_muon_config(rows, cols, batch=1, steps=5, coefficients=(3.4445, -4.7750, 2.0315),
                     momentum=0.95, nesterov=True, weight_decay=0.0, scale=1.0,
                     flags=0) -> mlpb_muon_config:
    return mlpb_muon_config(batch, rows, cols, steps, 1 if nesterov else 0,
                            (ctypes.c_float * 3)(*coefficients), momentum, weight_decay, scale,
                            flags)


def mlpb_muon_create(cfg: mlpb_muon_config) -> MuonHandle:
    """An orthogonalised update's handle on the current CUDA device."""
    lib, h, n = load_library(), ctypes.c_void_p(), ctypes.c_size_t()
    _check(lib.mlpb_muon_create(ctypes.byref(cfg), ctypes.byref(h)), "mlpb_muon_create")
    _check(lib.mlpb_muon_workspace_size(h.value, ctypes.byref(n)), "mlpb_muon_workspace_size")
    return MuonHandle(h.value, cfg, torch.cuda.current_device(), n.value)


def mlpb_muon_destroy(h: MuonHandle):
    if h is not None and h.ptr:
        load_library().mlpb_muon_destroy(h.ptr)
        h.ptr = 0


def mlpb_muon_workspace_size(h: MuonHandle) -> int:
    return h.workspace_bytes


def _muon_shape(h, t, name):
    """(device, shape) of a call's tensors: [rows][cols] matrices in any number of leading
    dimensions that make up the batch."""
    dev, c = _cuda_index(t, name), h.cfg
    if dev != h.device:
        raise ValueError(f"{name}: on cuda:{dev}, the handle on cuda:{h.device}")
    if t.dim() < 2 or tuple(t.shape[-2:]) != (c.rows, c.cols) \
            or t.numel() != c.batch * c.rows * c.cols:
        raise ValueError(f"{name}: expected {c.batch} matrices of shape {(c.rows, c.cols)}, "
                         f"got {tuple(t.shape)}")
    return dev, t.shape


def mlpb_muon_orthogonalize(h, U, O, workspace, stream=None):
    """O (bf16) from U (bf16 or fp32), both [..., rows, cols] (include/mlpb.h)."""
    dev, shape = _muon_shape(h, U, "U")
    if U.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"U: expected bfloat16 or float32, got {U.dtype}")
    args = [h.ptr, _arg(U, U.dtype, shape, "U", dev), 1 if U.dtype == torch.float32 else 0,
            _arg(O, torch.bfloat16, shape, "O", dev), _workspace(workspace, h.workspace_bytes, dev)]
    _call_on(dev, "mlpb_muon_orthogonalize", args, stream)


def mlpb_muon_step(h, G, M, W, lr, workspace, Wb=None, stream=None):
    """The momentum M and the weight W (fp32, in place) for the gradient G, and W in bf16 unless Wb
    is None; lr a CUDA tensor of one fp32."""
    dev, shape = _muon_shape(h, W, "W")
    f32 = torch.float32
    args = [h.ptr, _arg(G, f32, shape, "G", dev), _arg(M, f32, shape, "M", dev),
            _arg(W, f32, shape, "W", dev), _arg(Wb, torch.bfloat16, shape, "Wb", dev),
            _arg(lr, f32, (1,), "lr", dev), _workspace(workspace, h.workspace_bytes, dev)]
    _call_on(dev, "mlpb_muon_step", args, stream)


def mlpb_muon_last_device_error(h: MuonHandle, stream=None) -> int:
    """The status code (MLPB_OK, MLPB_ETIMEOUT, MLPB_ECUDA) without raising."""
    return _on_device(h.device, load_library().mlpb_muon_last_device_error, [h.ptr], stream)


def mlpb_last_device_error(h: Handle, stream=None) -> int:
    """Returns the status code (MLPB_OK, MLPB_ETIMEOUT, MLPB_ECUDA) without raising."""
    return load_library().mlpb_last_device_error(h.ptr, _stream(stream))


def mlpb_enable_timing(h: Handle, enable: bool = True):
    _check(load_library().mlpb_enable_timing(h.ptr, 1 if enable else 0), "mlpb_enable_timing")


def mlpb_read_timings(h: Handle, capacity: int = 64):
    buf = (mlpb_kernel_time * capacity)()
    n = ctypes.c_int()
    _check(load_library().mlpb_read_timings(h.ptr, buf, capacity, ctypes.byref(n)),
           "mlpb_read_timings")
    return [dict(name=buf[i].name.decode(), ms=buf[i].ms, flops=buf[i].flops,
                 bytes=buf[i].bytes, kernels=buf[i].kernels) for i in range(n.value)]


def mlpb_bias_grad_noalloc(inp, out, stream=None):
    """Column sums of a bf16 [rows][cols] CUDA tensor into the fp32 [cols] tensor `out`,
    with no device allocation (the library's fixed scratch array; see include/mlpb.h)."""
    rows, cols = inp.shape
    args = [_ptr(inp, torch.bfloat16, None, "in"), rows, cols,
            _ptr(out, torch.float32, (cols,), "out")]
    if out.device != inp.device:
        raise ValueError(f"in is on {inp.device} but out on {out.device}")
    # the library picks its scratch array and SM count from the current device, and the
    # stream must belong to that device too: make the tensors' device current
    with torch.cuda.device(inp.device):
        _check(load_library().mlpb_bias_grad_noalloc(*args, _stream(stream)),
               "mlpb_bias_grad_noalloc")


class MLPBlock:
    """Owns a handle plus the saved-activation and workspace buffers of one block shape.

    Convenience for callers that let torch allocate: forward() returns Y, backward()
    returns the gradient dict.  The arithmetic all happens in libmlpb.
    """

    def __init__(self, tokens, hidden, ffn, tp, act="gelu", has_bias=True,
                 seq_parallel_ln=False, ln_eps=1e-5, flags=0, device="cuda"):
        self.cfg = make_config(tokens, hidden, ffn, tp, act, has_bias, seq_parallel_ln, ln_eps,
                               flags)
        self.handle = mlpb_create(self.cfg)
        self.device = torch.device(device)
        self.act = act
        z_dtype, z_shape = _saved_z(self.handle)
        self.Z = torch.empty(z_shape, dtype=z_dtype, device=self.device)
        self.A = torch.empty((tokens, ffn), dtype=torch.bfloat16, device=self.device)
        self.workspace = torch.empty(mlpb_workspace_size(self.handle), dtype=torch.uint8,
                                     device=self.device)

    def close(self):
        mlpb_destroy(self.handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, X, W1, b1, W2, b2, Y=None, stream=None):
        if Y is None:
            Y = torch.empty((self.cfg.tokens, self.cfg.hidden), dtype=out_dtype(self.cfg),
                            device=self.device)
        mlpb_forward(self.handle, X, W1, b1, W2, b2, Y, self.Z, self.A, self.workspace, stream)
        return Y

    def alloc_grads(self, W1, W2):
        """dX plus the parameter-gradient buffers; zeroed main-grad buffers when the handle
        accumulates (MLPB_FLAG_ACCUMULATE_GRADS)."""
        c = self.cfg
        has_b = bool(c.has_bias)
        new = torch.zeros if c.flags & MLPB_FLAG_ACCUMULATE_GRADS else torch.empty
        f32 = dict(dtype=torch.float32, device=self.device)
        return dict(
            dX=torch.empty((c.tokens, c.hidden), dtype=out_dtype(c), device=self.device),
            dW1=new(W1.shape, **f32),
            dW2=new(W2.shape, **f32),
            db1=new((c.ffn,), **f32) if has_b else None,
            db2=new((c.hidden,), **f32) if has_b else None,
        )

    def backward(self, X, W1, W2, dY, grads=None, stream=None):
        g = grads if grads is not None else self.alloc_grads(W1, W2)
        mlpb_backward(self.handle, X, W1, W2, self.Z, self.A, dY, g["dX"], g["dW1"], g["dW2"],
                      g["db1"], g["db2"], self.workspace, stream)
        return g


class MLPBranch(MLPBlock):
    """The sequence-parallel pre-norm MLP branch Y = X + MLP(LN(X)) of one shape: an
    MLPBlock whose handle has the LayerNorm enabled, plus the saved Xn, mean and rstd."""

    def __init__(self, tokens, hidden, ffn, tp, act="gelu", has_bias=True, ln_eps=1e-5,
                 flags=0, device="cuda"):
        super().__init__(tokens, hidden, ffn, tp, act, has_bias, True, ln_eps, flags, device)
        self.Xn = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=self.device)
        self.mean = torch.empty((tokens,), dtype=torch.float32, device=self.device)
        self.rstd = torch.empty((tokens,), dtype=torch.float32, device=self.device)

    def forward(self, X, gamma, beta, W1, b1, W2, b2, Y=None, stream=None):
        if Y is None:
            Y = torch.empty((self.cfg.tokens, self.cfg.hidden), dtype=out_dtype(self.cfg),
                            device=self.device)
        mlpb_branch_forward(self.handle, X, gamma, beta, W1, b1, W2, b2, Y, self.Xn, self.mean,
                            self.rstd, self.Z, self.A, self.workspace, stream)
        return Y

    def alloc_grads(self, W1, W2):
        g = super().alloc_grads(W1, W2)
        new = torch.zeros if self.cfg.flags & MLPB_FLAG_ACCUMULATE_GRADS else torch.empty
        g["dgamma"] = new((self.cfg.hidden,), dtype=torch.float32, device=self.device)
        g["dbeta"] = new((self.cfg.hidden,), dtype=torch.float32, device=self.device)
        return g

    def backward(self, X, gamma, W1, W2, dY, grads=None, stream=None):
        g = grads if grads is not None else self.alloc_grads(W1, W2)
        mlpb_branch_backward(self.handle, X, gamma, W1, W2, self.Xn, self.mean, self.rstd, self.Z,
                             self.A, dY, g["dX"], g["dW1"], g["dW2"], g["db1"], g["db2"],
                             g["dgamma"], g["dbeta"], self.workspace, stream)
        return g


class ActCheckpoint8:
    """An activation whose input is kept for the backward as 8-bit codes: save() in the
    forward returns A = act(Z), grad() in the backward returns dZ and A again.  Owns the codes
    and scales of one [tokens][ffn] activation (tp shards), the only memory that has to live
    between the two."""

    def __init__(self, tokens, ffn, tp=1, act="gelu", device="cuda"):
        self.tokens, self.ffn, self.tp, self.act = tokens, ffn, tp, act
        self.device = _device(device)
        self.width = 2 * ffn if act == "swiglu" else ffn
        self.codes = torch.empty((tokens, self.width), dtype=torch.int8, device=self.device)
        self.scales = torch.empty((tokens, mlpb_act8_scales(act, ffn, tp)), dtype=torch.uint8,
                                  device=self.device)

    def _new(self, width):
        return torch.empty((self.tokens, width), dtype=torch.bfloat16, device=self.device)

    def save(self, Z, A=None, stream=None):
        if A is None:
            with _on(stream, self.device):
                A = self._new(self.ffn)
        mlpb_act8_save(self.act, Z, A, self.codes, self.scales, self.tp, stream)
        return A

    def grad(self, dA, dZ=None, A=None, codes=None, scales=None, stream=None):
        """(dZ, A); codes and scales other than the ones this object holds may be given."""
        with _on(stream, self.device):
            dZ = self._new(self.width) if dZ is None else dZ
            A = self._new(self.ffn) if A is None else A
        mlpb_act8_grad(self.act, dA, self.codes if codes is None else codes,
                       self.scales if scales is None else scales, dZ, A, self.tp, stream)
        return dZ, A


class Join:
    """The join between two blocks of one shape: forward() returns (Xout, Xn, stats),
    backward() the gradient dict.  Owns the backward's workspace."""

    def __init__(self, tokens, hidden, post_norm="none", pre_norm="none", gate_groups=0, eps=1e-5,
                 stream_dtype=torch.bfloat16, block_dtype=torch.bfloat16, accumulate=False,
                 has_block=True, device="cuda"):
        self.cfg = make_join_config(tokens, hidden, post_norm, pre_norm, gate_groups, eps,
                                    stream_dtype, block_dtype, accumulate, has_block)
        self.device = _device(device)
        self.workspace = torch.empty(_join_ws(self.cfg, self.device), dtype=torch.uint8,
                                     device=self.device)
        self._stream_dtype, self._has_block = stream_dtype, bool(has_block)
        self._has_pre = self.cfg.pre_norm != MLPB_NORM_NONE
        self._shape, self._stats = (tokens, hidden), (tokens, 4)

    def _rows(self, dtype):
        return torch.empty(self._shape, dtype=dtype, device=self.device)

    def forward(self, X, Y=None, res_scale=None, gate=None, gamma_post=None, beta_post=None,
                gamma_pre=None, beta_pre=None, Xout=None, Xn=None, stats=None, stream=None):
        """(Xout, Xn, stats); Xout is None without a block, Xn without a pre norm.  Pass the
        stream X itself as Xout to update it in place."""
        with _on(stream, self.device):
            if Xout is None and self._has_block:
                Xout = self._rows(self._stream_dtype)
            if Xn is None and self._has_pre:
                Xn = self._rows(torch.bfloat16)
            if stats is None:
                stats = torch.empty(self._stats, dtype=torch.float32, device=self.device)
        mlpb_join_fwd(self.cfg, X, Y, res_scale, gate, gamma_post, beta_post, gamma_pre, beta_pre,
                      Xout, Xn, stats, stream)
        return Xout, Xn, stats

    def alloc_grads(self, res_scale=False):
        """Gradient buffers: dX, dY and the parameters' (zeroed when they accumulate)."""
        c = self.cfg
        new = torch.zeros if c.flags & MLPB_JOIN_ACCUMULATE_GRADS else torch.empty

        def par(on, *shape):
            return new(shape, dtype=torch.float32, device=self.device) if on else None
        H, layer = c.hidden, MLPB_NORM_LAYER
        return dict(
            dX=self._rows(_join_types(c)[0]),
            dY=self._rows(torch.bfloat16) if c.has_block else None,
            dres_scale=par(res_scale, 1), dgate=par(c.gate_groups > 0, c.gate_groups, H),
            dgamma_post=par(c.post_norm != MLPB_NORM_NONE, H),
            dbeta_post=par(c.post_norm == layer, H),
            dgamma_pre=par(c.pre_norm != MLPB_NORM_NONE, H),
            dbeta_pre=par(c.pre_norm == layer, H))

    def backward(self, X, Y, Xout, stats, dXout, dXn=None, res_scale=None, gate=None,
                 gamma_post=None, beta_post=None, gamma_pre=None, beta_pre=None, grads=None,
                 stream=None):
        """The gradients for dXout (None: zero) and dXn of forward()'s outputs; X and Y may be
        None where the backward does not read them (include/mlpb.h).  `grads`: an alloc_grads()
        to write into again (half of a small call's host time is its allocations)."""
        g = grads
        if g is None:
            with _on(stream, self.device):
                g = self.alloc_grads(res_scale is not None)
        mlpb_join_bwd(self.cfg, X, Y, Xout, stats, res_scale, gate, gamma_post, beta_post,
                      gamma_pre, dXout, dXn, g["dX"], g["dY"], g["dres_scale"], g["dgate"],
                      g["dgamma_post"], g["dbeta_post"], g["dgamma_pre"], g["dbeta_pre"],
                      self.workspace, stream)
        return g


class MoEDecode:
    """A mixture-of-experts MLP for up to max_tokens (64) tokens: forward() returns (Y, ids,
    weights).  Owns a handle and its workspace."""

    def __init__(self, max_tokens, hidden, ffn, experts, topk, act="swiglu", normalize=True,
                 device="cuda"):
        self.cfg = make_moe_config(max_tokens, hidden, ffn, experts, topk, act, normalize)
        self.device = _device(device)
        with torch.cuda.device(self.device):
            self.handle = mlpb_moe_create(self.cfg)
        self.workspace = torch.empty(mlpb_moe_workspace_size(self.handle), dtype=torch.uint8,
                                     device=self.device)

    def close(self):
        mlpb_moe_destroy(self.handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, X, Wr, W1, W2, Y=None, ids=None, weights=None, stream=None):
        T, c = X.shape[0], self.cfg
        with _on(stream, self.device):
            if Y is None:
                Y = torch.empty((T, c.hidden), dtype=torch.bfloat16, device=self.device)
            if ids is None:
                ids = torch.empty((T, c.topk), dtype=torch.int32, device=self.device)
            if weights is None:
                weights = torch.empty((T, c.topk), dtype=torch.float32, device=self.device)
        mlpb_moe_forward(self.handle, X, Wr, W1, W2, Y, ids, weights, self.workspace, stream)
        return Y, ids, weights


class Linear8:
    """A linear layer y = x W^T on E4M3 operands with a scale for each block of 128, for up to
    max_tokens rows.  load() lays the weight out (before anything else, and again after each
    update); forward() and backward() as in include/mlpb.h.  Owns the weight's codes (with `training`, its transpose's
    too), what a forward keeps of X for the backward, and the workspace."""

    def __init__(self, max_tokens, inputs, outputs, training=True, out_dtype=torch.bfloat16,
                 device="cuda", flags=0):
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"out_dtype: bfloat16 or float32, not {out_dtype}")
        self.handle = None
        self._inputs, self._outputs = inputs, outputs
        self.cfg = mlpb_linear8_config(max_tokens, inputs, outputs, flags | (
            MLPB_LINEAR8_OUT_F32 if out_dtype == torch.float32 else 0))
        self.device, self.training, self.out_dtype = _device(device), training, out_dtype
        with torch.cuda.device(self.device):
            self.handle = mlpb_linear8_create(self.cfg)
        self.workspace = torch.empty(self.handle.workspace_bytes, dtype=torch.uint8,
                                     device=self.device)
        self.Wq = b128_empty(outputs, inputs, self.device)
        self.Wt = b128_empty(inputs, outputs, self.device) if training else None
        self._loaded = False  # Wq and Wt hold a weight
        self._saved = None  # X^T of the last forward that was given no Xt
        self._tokens = None  # of the last forward; None after one whose X^T lies in a given Xt
        if training:  # one buffer for any number of tokens
            ld, n = mlpb_b128_sizes(inputs, max_tokens)
            self._saved = torch.empty(inputs * ld + n, dtype=torch.uint8, device=self.device)

    def close(self):
        mlpb_linear8_destroy(self.handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load(self, W, stream=None):
        """Quantizes the weight W [outputs][inputs] (bf16 or fp32) in blocks of 128 x 128."""
        if tuple(W.shape) != (self.cfg.outputs, self.cfg.inputs):
            raise ValueError(f"W: expected shape {(self.cfg.outputs, self.cfg.inputs)}, "
                             f"got {tuple(W.shape)}")
        mlpb_b128_quantize(W, self.Wq, self.Wt, True, stream)
        self._loaded = True

    def _check_loaded(self):
        if not self._loaded:
            raise ValueError("Linear8: no weight yet, load() comes first")

    def saved(self, tokens):
        """The (codes, scales) of X^T that forward() without an Xt writes for this many tokens."""
        ld, n = mlpb_b128_sizes(self.cfg.inputs, tokens)
        m = self.cfg.inputs * ld
        return self._saved[:m].view(self.cfg.inputs, ld), self._saved[m:m + n]

    def _saved_args(self, tokens, Xt):
        """Pointers of the X^T that a call writes or reads: a given one, or this object's."""
        if Xt is not None:
            return _b128_args(Xt, self._inputs, tokens, "Xt", self.device.index)
        p = self._saved.data_ptr()  # as saved(), without its views
        return [p, p + self._inputs * ((tokens + 15) // 16 * 16)]

    def forward(self, X, Y=None, Xt=None, stream=None):
        """Y [tokens][outputs].  With `training`, Xt (or this object) receives X^T for the
        backward."""
        h, K, N = self.handle, self._inputs, self._outputs
        dev, T = _linear8_rows(h, X, K, "X")
        self._check_loaded()
        if Y is None:
            Y = _new((T, N), self.out_dtype, self.device, stream)
        args = [h.ptr, T, _arg(X, torch.bfloat16, (T, K), "X", dev),
                self.Wq[0].data_ptr(), self.Wq[1].data_ptr(),
                _arg(Y, self.out_dtype, (T, N), "Y", dev),
                *(self._saved_args(T, Xt) if Xt is not None or self.training else (None, None)),
                self.workspace.data_ptr()]
        _call_on(dev, "mlpb_linear8_forward", args, stream)
        self._tokens = T if Xt is None else None
        return Y

    def backward(self, dY, dX=None, dW=None, Xt=None, accumulate=False, input_grad=True,
                 weight_grad=True, stream=None):
        """(dX, dW) for the rows of the last forward, or for an Xt that a forward wrote (after a
        forward with an Xt it has to be named; saved() is what the one before left here); with
        `accumulate` dW is added into; without `input_grad` or `weight_grad` dX or dW, unless it is
        given, is None and not computed (dX alone takes no rows of a forward).  A captured forward
        counts as it is captured, not as it is replayed."""
        if not self.training:
            raise ValueError("Linear8: made with training=False")
        weight_grad = weight_grad or dW is not None
        if not (input_grad or weight_grad or dX is not None):
            raise ValueError("input_grad, weight_grad: neither gradient is asked for")
        if accumulate and dW is None:
            raise ValueError("dW: nothing given to add into")
        h, K, N = self.handle, self._inputs, self._outputs
        dev, T = _linear8_rows(h, dY, N, "dY")
        self._check_loaded()
        if Xt is None and weight_grad and T > 0 and T != self._tokens:
            if self._tokens is None:
                raise ValueError("Xt: not given, and the last forward kept no rows here")
            raise ValueError(f"dY: {T} tokens, the last forward had {self._tokens}")
        if dX is None and input_grad:
            dX = _new((T, K), self.out_dtype, self.device, stream)
        if dW is None and weight_grad:
            dW = _new((N, K), torch.float32, self.device, stream)
        args = [h.ptr, T, _arg(dY, torch.bfloat16, (T, N), "dY", dev),
                self.Wt[0].data_ptr(), self.Wt[1].data_ptr(),
                *(self._saved_args(T, Xt) if weight_grad else (None, None)),
                _arg(dX, self.out_dtype, (T, K), "dX", dev),
                _arg(dW, torch.float32, (N, K), "dW", dev),
                1 if accumulate else 0, self.workspace.data_ptr()]
        _call_on(dev, "mlpb_linear8_backward", args, stream)
        return dX, dW


class Muon:
    """The orthogonalised update of `batch` matrices [rows][cols], each by itself: orthogonalize()
    alone, or step() with momentum, decay and the weight's update.  The shards of a weight as a
    batch (dW1 [t][2][Fs][H] is 2 t matrices) are the blockwise update; that of the whole weight
    takes whole matrices (include/mlpb.h).  Owns a handle and its workspace."""

    def __init__(self, rows, cols, batch=1, steps=5, coefficients=(3.4445, -4.7750, 2.0315),
                 momentum=0.95, nesterov=True, weight_decay=0.0, scale=1.0, device="cuda",
                 flags=0):
        self.handle = None
        self.cfg = make_muon_config(rows, cols, batch, steps, coefficients, momentum, nesterov,
                                    weight_decay, scale, flags)
        self.device = _device(device)
        with torch.cuda.device(self.device):
            self.handle = mlpb_muon_create(self.cfg)
        self.workspace = torch.empty(self.handle.workspace_bytes, dtype=torch.uint8,
                                     device=self.device)

    def close(self):
        mlpb_muon_destroy(self.handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def orthogonalize(self, U, O=None, stream=None):
        """O, bf16 in the shape of U (bf16 or fp32)."""
        if O is None:
            O = _new(U.shape, torch.bfloat16, self.device, stream)
        mlpb_muon_orthogonalize(self.handle, U, O, self.workspace, stream)
        return O

    def step(self, W, M, G, lr, Wb=None, stream=None):
        """Updates the momentum M and the weight W (fp32) in place for the gradient G; Wb, if
        given, receives W in bf16.  lr: a CUDA tensor of one fp32."""
        mlpb_muon_step(self.handle, G, M, W, lr, self.workspace, Wb, stream)
