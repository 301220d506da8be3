"""Pins of the mixture-of-experts oracle (CPU), and the entry points' refusals, which return
before the device is touched."""
import ctypes

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from megatron_tensor_transformer_tma_gb300 import build as mbuild
from oracle import mlp as omlp
from oracle import moe


def _draw(T=5, H=16, F=8, E=6, act="swiglu", seed=0):
    n = np.random.default_rng(seed).standard_normal
    return n((T, H)), n((E, H)), n((E, 2, F, H) if act == "swiglu" else (E, F, H)), n((E, H, F))


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_all_experts_with_equal_weights_are_the_mean_of_mlps(act):
    X, Wr, W1, W2 = _draw(act=act)
    _, ids, w = moe.route(X, 0 * Wr, 6, False)
    assert np.array_equal(ids, np.tile(np.arange(6), (5, 1)))   # equal logits: by index
    assert np.allclose(w, 1 / 6)
    Y = moe.forward(X, W1, W2, ids, w, act)
    ref = sum(omlp.mlp_forward(X, W1[e][None], None, W2[e][None], None, act)["Y"]
              for e in range(6)) / 6
    assert np.abs(Y - ref).max() < 1e-12


def test_one_expert_is_the_mlp():
    X, Wr, W1, W2 = _draw(E=1)
    for norm in (False, True):
        _, ids, w = moe.route(X, Wr, 1, norm)
        assert (ids == 0).all() and (w == 1).all()
    ref = omlp.mlp_forward(X, W1, None, W2, None, "swiglu")["Y"]
    assert np.abs(moe.forward(X, W1, W2, ids, w, "swiglu") - ref).max() < 1e-12


def test_routing_by_brute_force():
    X, Wr, _, _ = _draw(T=40, E=9)
    l, ids, w = moe.route(X, Wr, 4, False)
    lt = torch.from_numpy(l)
    assert np.array_equal(ids, lt.topk(4).indices.numpy())
    assert np.allclose(w, torch.softmax(lt, 1).gather(1, torch.from_numpy(ids)).numpy())
    assert np.allclose(moe.route(X, Wr, 4, True)[2].sum(1), 1.0)


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mlpb.load_library()


def _create(lib, **kw):
    args = dict(max_tokens=4, hidden=64, ffn=32, experts=8, topk=2)
    args.update(kw)
    h = ctypes.c_void_p()
    st = lib.mlpb_moe_create(ctypes.byref(mlpb.make_moe_config(**args)), ctypes.byref(h))
    if st == mlpb.MLPB_OK:
        lib.mlpb_moe_destroy(h)
    else:
        assert not h.value
    return st


@pytest.mark.parametrize("kw", [
    dict(max_tokens=0), dict(hidden=0), dict(ffn=-8), dict(experts=0), dict(topk=0),
    dict(topk=9), dict(flags=1)])
def test_config_refused_as_invalid(lib, kw):
    assert _create(lib, **kw) == mlpb.MLPB_EINVAL


@pytest.mark.parametrize("kw", [
    dict(max_tokens=65), dict(hidden=60), dict(ffn=12), dict(experts=257),
    dict(experts=32, topk=17), dict(hidden=(1 << 20) + 8), dict(ffn=(1 << 20) + 8)])
def test_config_refused_as_unsupported(lib, kw):
    assert _create(lib, **kw) == mlpb.MLPB_EUNSUPPORTED


def test_other_refusals(lib):
    E = mlpb.MLPB_EINVAL
    assert _create(lib) in (mlpb.MLPB_OK, mlpb.MLPB_ECUDA)
    c = mlpb.make_moe_config(4, 64, 32, 8, 2)
    h = ctypes.c_void_p()
    assert lib.mlpb_moe_create(None, ctypes.byref(h)) == E
    assert lib.mlpb_moe_create(ctypes.byref(c), None) == E
    for field, value in (("act", 2), ("normalize", 2)):
        bad = mlpb.make_moe_config(4, 64, 32, 8, 2)
        setattr(bad, field, value)
        assert lib.mlpb_moe_create(ctypes.byref(bad), ctypes.byref(h)) == E
    n = ctypes.c_size_t()
    assert lib.mlpb_moe_workspace_size(None, ctypes.byref(n)) == E
    assert lib.mlpb_moe_forward(None, 1, *[0x10000] * 8, None) == E
    assert lib.mlpb_moe_last_device_error(None, None) == E
    lib.mlpb_moe_destroy(None)
    with pytest.raises(KeyError):
        mlpb.make_moe_config(4, 64, 32, 8, 2, act="relu")
