"""Pins of the 8-bit checkpoint oracle (CPU): its codes against the definition's inequalities
and torch's own rounding, its gradients against differences; and the entry points' refusals,
which return before the device is touched."""
import ctypes

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from megatron_tensor_transformer_tma_gb300 import build as mbuild
from oracle import act8
from oracle import mlp as omlp

SHAPES = [(3, 8, 1, "gelu"), (2, 72, 1, "gelu"), (4, 80, 2, "swiglu"), (2, 192, 3, "swiglu")]


def _z(T, F, tp, act, seed=0):
    g = torch.Generator().manual_seed(seed)
    f1 = 2 * F if act == "swiglu" else F
    return (1.3 * torch.randn(T, f1, generator=g)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("T,F,tp,act", SHAPES)
def test_codes_satisfy_the_definition(T, F, tp, act):
    z = _z(T, F, tp, act)
    z[0, :8] = 0.0
    codes, scales = act8.quantize(z, F, tp, act)
    zh = act8.decode(codes, scales, F, tp, act)
    n, width = act8.segments(F, tp, act)
    for s in range(n):
        for b in range(-(-width // 32)):
            sl = slice(s * width + 32 * b, s * width + min(width, 32 * b + 32))
            step = np.ldexp(1.0, scales[:, s * -(-width // 32) + b].astype(int) - 127)[:, None]
            amax = np.abs(z[:, sl]).max(1, keepdims=True)
            assert (amax <= 127 * step).all()
            nz = amax > 0
            assert (amax[nz] > 127 * step[nz] / 2).all()    # the next finer step would not do
            assert (np.abs(zh[:, sl] - z[:, sl]) <= step / 2).all()
            want = torch.round(torch.from_numpy(z[:, sl] / step)).numpy()  # ties to even
            assert np.array_equal(codes[:, sl].astype(float), want)


def test_extreme_blocks():
    z = np.zeros((6, 32))
    z[1, 3] = 2.0 ** -133                 # the smallest bf16: the step stays 2^-126
    z[2, 0], z[2, 1] = 127.0, 126.5       # exactly at the border, and a tie to even
    z[3, 0] = 127.5                       # bf16 127.5 does not fit 127 steps of 1
    z[4, 0] = np.inf
    z[5, 7] = np.nan
    codes, scales = act8.quantize(z, 32, 1, "gelu")
    assert scales[:, 0].tolist() == [127, 1, 127, 128, 255, 255]
    assert codes[0].any() == 0 and codes[2, 0] == 127 and codes[2, 1] == 126
    assert codes[3, 0] == 64
    assert np.isnan(act8.decode(codes, scales, 32, 1, "gelu")[4:]).all()


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_gradient_against_differences(act):
    F, tp = 16, 2
    z = _z(3, F, tp, act, 1)
    dA = np.random.default_rng(2).standard_normal((3, F))
    g = act8.act_grad(dA, z, F, tp, act)
    h = 1e-6
    for i in range(z.shape[1]):
        e = np.zeros_like(z)
        e[:, i] = h
        d = ((act8.act(z + e, F, tp, act) - act8.act(z - e, F, tp, act)) * dA).sum(1) / (2 * h)
        assert np.allclose(g[:, i], d, atol=1e-8, rtol=1e-6)


def test_gelu_form():
    """The oracle's GELU is the block oracle's, where that one's tanh form keeps its digits."""
    z = np.linspace(-8, 8, 4001)
    assert np.abs(act8.gelu(z) - omlp.gelu_tanh(z)).max() < 1e-14
    assert np.abs(act8.gelu_grad(z) - omlp.gelu_tanh_grad(z)).max() < 1e-13


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mlpb.load_library()


def test_scales_per_row(lib):
    assert mlpb.mlpb_act8_scales("gelu", 40, 5) == 2
    assert mlpb.mlpb_act8_scales("swiglu", 1032, 3) == 6 * 11
    assert mlpb.mlpb_act8_scales("swiglu", 64, 8) == 16


def test_refusals_before_the_device(lib):
    E, U = mlpb.MLPB_EINVAL, mlpb.MLPB_EUNSUPPORTED
    a, b, c = 0x10000, 0x20000, 0x30001  # stand-ins that validation never dereferences
    for fn, args in ((lib.mlpb_act8_save, [a, b, a, c]), (lib.mlpb_act8_grad, [a, b, c, a, b])):
        assert fn(2, 4, 64, 1, *args, None) == E        # no such activation
        assert fn(0, -1, 64, 1, *args, None) == E
        assert fn(0, 4, 0, 1, *args, None) == E
        assert fn(0, 4, 64, 0, *args, None) == E
        assert fn(1, 4, 64, 3, *args, None) == U        # F % tp
        assert fn(0, 4, 24, 2, *args, None) == U        # (F/tp) % 8
        assert fn(0, 4, 1 << 29, 1, *args, None) == U   # features past the index range
        assert fn(0, 0, 64, 1, *([None] * len(args)), None) == mlpb.MLPB_OK
        for i in range(len(args)):
            bad = list(args)
            bad[i] = None
            optional = i == (1 if fn is lib.mlpb_act8_save else 4)
            if not optional:
                assert fn(0, 4, 64, 1, *bad, None) == E
            if args[i] != c:
                bad[i] = args[i] + 8
                assert fn(0, 4, 64, 1, *bad, None) == E  # misaligned
    n = ctypes.c_int64()
    assert lib.mlpb_act8_scales(0, 64, 1, None) == E
    assert lib.mlpb_act8_scales(0, 60, 1, ctypes.byref(n)) == U


def test_binding_refuses(lib):
    z = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mlpb.mlpb_act8_save("gelu", z, None, z, z)
    with pytest.raises(TypeError):
        mlpb.mlpb_act8_grad("gelu", None, z, z, z)
    with pytest.raises(KeyError):
        mlpb.mlpb_act8_scales("relu", 64)


def test_checkpoint_flag_validation(lib):
    def create(**kw):
        args = dict(tokens=128, hidden=256, ffn=1024, tp=2, act="gelu", has_bias=True)
        args.update(kw)
        h = ctypes.c_void_p()
        st = lib.mlpb_create(ctypes.byref(mlpb.make_config(**args)), ctypes.byref(h))
        if st == mlpb.MLPB_OK:
            lib.mlpb_destroy(h)
        return st
    C8 = mlpb.MLPB_FLAG_CHECKPOINT8
    ok = (mlpb.MLPB_OK, mlpb.MLPB_ECUDA)  # without a GPU a valid config ends at the device query
    assert create(flags=C8) in ok
    assert create(flags=C8 | mlpb.MLPB_FLAG_RECOMPUTE_ACT | mlpb.MLPB_FLAG_BF16_OUT) in ok
    assert create(flags=C8, ffn=2 * 48) == mlpb.MLPB_EUNSUPPORTED   # Fs % 32
    assert create(flags=C8 | mlpb.MLPB_FLAG_FP8) == mlpb.MLPB_EUNSUPPORTED
    src = open(mbuild.INCLUDE + "/mlpb.h").read()
    assert "#define MLPB_FLAG_CHECKPOINT8 0x100u" in src
