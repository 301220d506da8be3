"""Pins of the block-scaled E4M3 oracle: torch's own E4M3 conversion, the scale's inequality, the
layer's products against differences; and the library's refusals and sizes, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from megatron_tensor_transformer_tma_gb300 import build as mbuild
from oracle import b128


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mlpb.load_library()


def test_rounding_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(size=4000) * 2.0 ** -7,
                        b128.e4m3_values(), -b128.e4m3_values(),
                        (b128.e4m3_values()[1:] + b128.e4m3_values()[:-1]) / 2])
    x = torch.tensor(x, dtype=torch.float32)
    want = x.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(b128.round_e4m3(x.double().numpy()), want)


@pytest.mark.parametrize("square", [False, True])
def test_scales_use_the_range(square):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(130, 300)) * np.exp(4 * rng.normal(size=(130, 1)))
    x[5, :128] = 0
    v, s = b128.quantize(x, square)
    rows = 128 if square else 1
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = (slice(i * rows, (i + 1) * rows), slice(j * 128, (j + 1) * 128))
            top, k = np.abs(x[at]).max(), 127 - s[i, j]
            assert top == 0 and k == 0 or top * 2.0 ** k <= 448 < top * 2.0 ** (k + 1)
            # half a step of a normal value, or of the smallest
            err = np.abs(v[at] - x[at])
            assert (err <= np.maximum(np.abs(x[at]) * 2.0 ** -4, 2.0 ** (-10 - k))).all()


def test_range_of_scales():
    assert b128.scale_exponent(np.finfo(np.float32).max) == -120
    assert b128.scale_exponent(2.0 ** -149) == 126
    v, s = b128.quantize(np.array([[1.0, np.inf] + [0.0] * 126 + [2.0]]))
    assert np.isnan(v[0, :128]).all() and v[0, 128] == 2.0 and s[0, 0] == 255


def test_gradients_are_those_of_the_rounded_product():
    rng = np.random.default_rng(2)
    X, W, dY = rng.normal(size=(9, 40)), rng.normal(size=(24, 40)), rng.normal(size=(9, 24))
    o = b128.linear(X, W, dY)
    xq, wq, d = b128.quantize(X)[0], b128.quantize(W, True)[0], b128.quantize(dY)[0]
    i, j, h = 3, 17, 1e-6
    e = np.zeros_like(xq)
    e[i, j] = h  # the products are linear: differences of them are exact up to rounding
    assert np.isclose(((xq + e) @ wq.T * d).sum() - (xq @ wq.T * d).sum(), h * o["dX"][0][i, j],
                      rtol=1e-4)
    dt, xt = b128.quantize(dY.T)[0].T, b128.quantize(X.T)[0].T
    e = np.zeros_like(wq)
    e[5, j] = h
    assert np.isclose((xt @ (wq + e).T * dt).sum() - (xt @ wq.T * dt).sum(), h * o["dW"][0][5, j],
                      rtol=1e-4)


def test_sizes(lib):
    ld, n = ctypes.c_int64(), ctypes.c_size_t()
    for rows, cols, want in ((1, 1, (16, 512)), (128, 512, (512, 512)), (129, 513, (528, 2048)),
                             (0, 64, (64, 0)), (77, 1032, (1040, 1536))):
        assert lib.mlpb_b128_sizes(rows, cols, ctypes.byref(ld), ctypes.byref(n)) == mlpb.MLPB_OK
        assert (ld.value, n.value) == want
    assert lib.mlpb_b128_sizes(-1, 1, ctypes.byref(ld), ctypes.byref(n)) == mlpb.MLPB_EINVAL
    assert lib.mlpb_b128_sizes(1, 1, None, ctypes.byref(n)) == mlpb.MLPB_EINVAL
    assert lib.mlpb_b128_sizes(2 ** 21, 1, ctypes.byref(ld), ctypes.byref(n)) \
        == mlpb.MLPB_EUNSUPPORTED


def test_quantize_refuses(lib):
    E, U, q = mlpb.MLPB_EINVAL, mlpb.MLPB_EUNSUPPORTED, lib.mlpb_b128_quantize
    x, a, b, c, d = (0x10000 * i for i in range(1, 6))  # never dereferenced
    assert q(None, 0, 8, 8, 0, a, b, c, d, None) == E
    assert q(x, 2, 8, 8, 0, a, b, c, d, None) == E
    assert q(x, 0, 8, 8, 2, a, b, c, d, None) == E
    assert q(x, 0, -1, 8, 0, a, b, c, d, None) == E
    assert q(x, 0, 8, 12, 0, a, b, c, d, None) == U
    assert q(x, 0, 2 ** 20 + 1, 8, 0, a, b, c, d, None) == U
    assert q(x, 0, 8, 8, 0, None, None, None, None, None) == E
    assert q(x, 0, 8, 8, 0, a, None, c, d, None) == E
    assert q(x, 0, 8, 8, 0, a, b, None, d, None) == E
    for i in range(5):
        p = [x, a, b, c, d]
        p[i] += 8
        assert q(p[0], 0, 8, 8, 0, *p[1:], None) == E
    assert q(None, 0, 0, 8, 0, None, None, None, None, None) == mlpb.MLPB_OK


@pytest.mark.parametrize("kw,status", [
    (dict(max_tokens=0), mlpb.MLPB_EINVAL), (dict(inputs=0), mlpb.MLPB_EINVAL),
    (dict(outputs=-8), mlpb.MLPB_EINVAL), (dict(flags=0x4), mlpb.MLPB_EINVAL),
    (dict(inputs=12), mlpb.MLPB_EUNSUPPORTED), (dict(outputs=100), mlpb.MLPB_EUNSUPPORTED),
    (dict(max_tokens=2 ** 20 + 1), mlpb.MLPB_EUNSUPPORTED),
    (dict(inputs=2 ** 20 + 8), mlpb.MLPB_EUNSUPPORTED)])
def test_linear8_create_refuses(lib, kw, status):
    cfg = mlpb.mlpb_linear8_config(**{**dict(max_tokens=8, inputs=64, outputs=64, flags=0), **kw})
    h = ctypes.c_void_p()
    assert lib.mlpb_linear8_create(ctypes.byref(cfg), ctypes.byref(h)) == status
    assert not h.value


def test_linear8_null_arguments(lib):
    E, n = mlpb.MLPB_EINVAL, ctypes.c_size_t()
    assert lib.mlpb_linear8_create(None, None) == E
    assert lib.mlpb_linear8_workspace_size(None, ctypes.byref(n)) == E
    assert lib.mlpb_linear8_forward(None, 1, *[None] * 8) == E
    assert lib.mlpb_linear8_backward(None, 1, *[None] * 7, 0, None, None) == E
    assert lib.mlpb_linear8_last_device_error(None, None) == E
    lib.mlpb_linear8_destroy(None)


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mlpb.mlpb_b128_quantize(x, None, None)
    with pytest.raises(TypeError):
        mlpb.Linear8(4, 64, 64, out_dtype=torch.float16)


def test_header_flag_values_match_binding():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                            "include", "mlpb.h")).read()
    for name in ("MLPB_LINEAR8_OUT_F32", "MLPB_LINEAR8_FAULT_INJECT"):
        m = re.search(rf"#define\s+{name}\s+(0x[0-9a-fA-F]+)u", src)
        assert m and int(m.group(1), 16) == getattr(mlpb, name), name


@pytest.mark.parametrize("rows,cols", [(0, 64), (64, 0), (0, 0)])
def test_values_of_nothing(lib, rows, cols):
    v = mlpb.b128_values(mlpb.b128_empty(rows, cols, "cpu"), rows, cols)
    assert tuple(v.shape) == (rows, cols) and v.dtype == torch.float64
