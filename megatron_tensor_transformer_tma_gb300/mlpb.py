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
