"""Pins of the join's oracle (CPU): gradients against differences, the norms against the
LayerNorm oracle; and the entry points' refusals, which return before the device is touched."""
import ctypes

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from megatron_tensor_transformer_tma_gb300 import build as mbuild
from oracle import join
from oracle import layernorm as oln

EPS = 1e-3
KINDS = ["none", "layer", "rms"]


def _case(post, pre, groups, T=6, H=16, seed=0):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    return dict(X=2 * n((T, H)), Y=n((T, H)) + 0.3, alpha=0.7,
                gate=n((groups, H)) if groups else None, post=post, gamma_post=1 + 0.1 * n(H),
                beta_post=n(H), pre=pre, gamma_pre=1 + 0.1 * n(H), beta_pre=n(H), eps=EPS)


@pytest.mark.parametrize("post", KINDS)
@pytest.mark.parametrize("pre", KINDS)
@pytest.mark.parametrize("groups", [0, 1, 3, 6])
def test_gradients_against_differences(post, pre, groups):
    c = _case(post, pre, groups)
    r = np.random.default_rng(1)
    dXout, dXn = r.standard_normal((6, 16)), r.standard_normal((6, 16))

    def loss(**kw):
        o = join.forward(**{**c, **kw})
        return (o["Xout"] * dXout).sum() + ((o["Xn"] * dXn).sum() if pre != "none" else 0.0)

    f = join.forward(**c)
    args = {k: v for k, v in c.items() if k != "beta_pre"}
    g = join.backward(Xout=f["Xout"], dXout=dXout, dXn=dXn, **args)
    h = 1e-6
    assert abs((loss(alpha=0.7 + h) - loss(alpha=0.7 - h)) / (2 * h) - g["dres_scale"][0]) < 1e-6
    for name in ("X", "Y", "gate", "gamma_post", "beta_post", "gamma_pre", "beta_pre"):
        got = g.get("d" + name)
        if got is None:
            continue
        for i in np.random.default_rng(2).integers(0, c[name].size, 12):
            e = np.zeros(c[name].size)
            e[i] = h
            e = e.reshape(c[name].shape)
            d = (loss(**{name: c[name] + e}) - loss(**{name: c[name] - e})) / (2 * h)
            assert abs(d - got.reshape(-1)[i]) < 1e-6 * max(1.0, abs(d)), (name, i)


def test_layer_norm_is_the_layernorm_oracle():
    c = _case("none", "layer", 0)
    f = join.forward(**{**c, "Y": np.zeros_like(c["Y"]), "alpha": 1.0})
    ref = oln.layernorm_fwd(c["X"], c["gamma_pre"], c["beta_pre"], EPS)
    assert np.abs(f["Xn"] - ref[0]).max() < 1e-12


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mlpb.load_library()


def _cfg(**kw):
    args = dict(tokens=4, hidden=64, post_norm="rms", pre_norm="layer", gate_groups=2)
    args.update(kw)
    return mlpb.make_join_config(**args)


FWD = ["X", "Y", "alpha", "gate", "gpost", "bpost", "gpre", "bpre", "Xout", "Xn", "stats"]
BWD = ["X", "Y", "Xout", "stats", "alpha", "gate", "gpost", "bpost", "gpre", "dXout", "dXn", "dX",
       "dY", "dalpha", "dgate", "dgpost", "dbpost", "dgpre", "dbpre", "ws"]
GIVEN = {k: 0x10000 * (i + 1) for i, k in enumerate(dict.fromkeys(FWD + BWD))}


def _call(lib, which, cfg, **kw):
    """The status of a call with stand-in pointers, for calls that validation must refuse."""
    names = FWD if which == "fwd" else BWD
    a = {k: GIVEN[k] for k in names}
    a.update({k: None for k in ("bpost", "dbpost") if k in a})  # an RMS post norm has no beta
    a.update(kw)
    fn = lib.mlpb_join_fwd if which == "fwd" else lib.mlpb_join_bwd
    return fn(ctypes.byref(cfg), *[a[k] for k in names], None)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(hidden=0), dict(gate_groups=-1), dict(eps=0.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(has_block=False)])
def test_config_refused_as_invalid(lib, kw):
    n = ctypes.c_size_t()
    assert lib.mlpb_join_workspace_size(ctypes.byref(_cfg(**kw)), ctypes.byref(n)) \
        == mlpb.MLPB_EINVAL
    assert _call(lib, "fwd", _cfg(**kw)) == mlpb.MLPB_EINVAL
    assert _call(lib, "bwd", _cfg(**kw)) == mlpb.MLPB_EINVAL


@pytest.mark.parametrize("kw", [
    dict(hidden=60), dict(hidden=16392), dict(tokens=1 << 31), dict(gate_groups=3),
    dict(gate_groups=8)])
def test_config_refused_as_unsupported(lib, kw):
    for which in ("fwd", "bwd"):
        assert _call(lib, which, _cfg(**kw)) == mlpb.MLPB_EUNSUPPORTED


def test_config_enums_and_flags(lib):
    for field, value in (("post_norm", 3), ("pre_norm", -1), ("has_block", 2), ("flags", 8)):
        c = _cfg()
        setattr(c, field, value)
        assert _call(lib, "fwd", c) == mlpb.MLPB_EINVAL
    with pytest.raises(KeyError):
        _cfg(post_norm="batch")
    with pytest.raises(TypeError):
        _cfg(stream_dtype=torch.float16)
    assert lib.mlpb_join_fwd(None, *[None] * 12) == mlpb.MLPB_EINVAL
    assert lib.mlpb_join_bwd(None, *[None] * 21) == mlpb.MLPB_EINVAL
    assert lib.mlpb_join_workspace_size(ctypes.byref(_cfg()), None) == mlpb.MLPB_EINVAL


@pytest.mark.parametrize("which,names,optional", [
    ("fwd", FWD, {"alpha"}), ("bwd", BWD, {"dXout"})])
def test_pointers_refused(lib, which, names, optional):
    """Each pointer missing, misaligned, or given where the configuration has no use for it."""
    E = mlpb.MLPB_EINVAL
    for k in names:
        if k not in ("bpost", "dbpost"):
            if k not in optional:
                assert _call(lib, which, _cfg(), **{k: None}) == E, k
            off = 2 if k in ("alpha", "dalpha") else 8
            assert _call(lib, which, _cfg(), **{k: GIVEN[k] + off}) == E, k
        else:
            assert _call(lib, which, _cfg(), **{k: GIVEN[k]}) == E, k
    none = _cfg(gate_groups=0)
    assert _call(lib, which, none) == E                              # a gate without groups
    alone = _cfg(gate_groups=0, post_norm="none", has_block=False)
    assert _call(lib, which, alone, gate=None, gpost=None) == E      # a block where there is none
    if which == "bwd":
        assert _call(lib, which, _cfg(pre_norm="none"), gpre=None, dgpre=None, dbpre=None) == E
        assert _call(lib, which, _cfg(pre_norm="none"), gpre=None, dgpre=None, dbpre=None,
                     dXn=None, dXout=None) == E                      # no gradient at all


def test_binding_refuses(lib):
    with pytest.raises(TypeError):
        mlpb.mlpb_join_fwd(_cfg(), None, *[None] * 10)
    with pytest.raises(ValueError, match="CUDA"):
        mlpb.mlpb_join_fwd(_cfg(), torch.zeros(4, 64), *[None] * 10)
