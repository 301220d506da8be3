"""Pins of the orthogonalisation's oracle (singular values against products, orthogonality, signs,
the effect of the operands' rounding), and the library's refusals, without a GPU."""
import ctypes

import numpy as np
import pytest

import megatron_tensor_transformer_tma_gb300 as mlpb
from megatron_tensor_transformer_tma_gb300 import build as mbuild
from oracle import muon


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mlpb.load_library()


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (9, 1), (24, 40), (40, 24), (32, 32)])
def test_products_are_the_polynomials_of_the_singular_values(shape):
    U = np.random.default_rng(0).normal(size=shape)
    assert np.allclose(muon.orthogonalize(U), muon.by_products(U), atol=1e-12)
    assert np.allclose(muon.orthogonalize(U.T), muon.orthogonalize(U).T, atol=1e-12)
    assert np.allclose(muon.orthogonalize(-1e-3 * U), -muon.orthogonalize(U), atol=1e-12)


def test_singular_values_come_near_one():
    U = np.random.default_rng(1).normal(size=(48, 200))
    s = np.linalg.svd(muon.orthogonalize(U), compute_uv=False)
    assert 0.6 < s.min() and s.max() < 1.3
    # the cubic that converges: to the orthogonal factor itself
    O = muon.orthogonalize(U, 40, (1.5, -0.5, 0.0))
    assert np.allclose(O @ O.T, np.eye(48), atol=1e-9)
    P, _, Q = np.linalg.svd(U, full_matrices=False)
    assert np.allclose(O, P @ Q, atol=1e-9)


def test_a_zero_matrix_stays_zero():
    assert not muon.orthogonalize(np.zeros((3, 5))).any()


def test_rounded_operands_move_the_result_by_little():
    rng = np.random.default_rng(2)
    for U in (rng.normal(size=(96, 256)), rng.normal(size=(256, 96)),
              rng.normal(size=(96, 4)) @ rng.normal(size=(4, 128)) + 0.1 * rng.normal(size=(96, 128))):
        O = muon.orthogonalize(U)
        e = np.linalg.norm(muon.rounded(U) - O) / np.linalg.norm(O)
        assert 1e-6 < e < 2e-3


def test_step_without_momentum_or_decay_is_the_update():
    rng = np.random.default_rng(3)
    W, M, G = (rng.normal(size=(8, 12)) for _ in range(3))
    w, m, O, U = muon.step(W, M, G, 0.1, 0.0, True, 0.0, 2.0)
    assert np.allclose(m, G) and np.allclose(U, G)
    assert np.allclose(W - w, 0.2 * O)
    w, m, O, U = muon.step(W, M, G, 0.1, 0.5, False, 0.2, 1.0)
    assert np.allclose(U, 0.5 * M + G) and np.allclose(w, 0.98 * W - 0.1 * O)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), mlpb.MLPB_EINVAL), (dict(rows=0), mlpb.MLPB_EINVAL),
    (dict(cols=-1), mlpb.MLPB_EINVAL), (dict(steps=0), mlpb.MLPB_EINVAL),
    (dict(momentum=1.0), mlpb.MLPB_EINVAL), (dict(momentum=-0.1), mlpb.MLPB_EINVAL),
    (dict(momentum=float("nan")), mlpb.MLPB_EINVAL), (dict(scale=float("inf")), mlpb.MLPB_EINVAL),
    (dict(weight_decay=float("nan")), mlpb.MLPB_EINVAL), (dict(flags=2), mlpb.MLPB_EINVAL),
    (dict(coefficients=(float("nan"), 0, 0)), mlpb.MLPB_EINVAL),
    (dict(rows=65537), mlpb.MLPB_EUNSUPPORTED), (dict(cols=65537), mlpb.MLPB_EUNSUPPORTED),
    (dict(batch=65536), mlpb.MLPB_EUNSUPPORTED), (dict(steps=65), mlpb.MLPB_EUNSUPPORTED),
    (dict(batch=65535, rows=65536, cols=65536), mlpb.MLPB_EUNSUPPORTED),
    (dict(coefficients=(2.5, 0.0, 0.0)), mlpb.MLPB_EUNSUPPORTED),      # grows past 2
    (dict(coefficients=(1.0, -61.0, 61.0)), mlpb.MLPB_EUNSUPPORTED)])
def test_create_refuses(lib, kw, status):
    cfg = mlpb.make_muon_config(**{**dict(rows=64, cols=64), **kw})
    h = ctypes.c_void_p()
    assert lib.mlpb_muon_create(ctypes.byref(cfg), ctypes.byref(h)) == status
    assert not h.value


@pytest.mark.parametrize("coef", [(3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375),
                                  (2.0, -1.5, 0.5)])
def test_usual_coefficients_pass_the_host_checks(lib, coef):
    """Without a GPU a valid configuration fails at the device query alone."""
    cfg = mlpb.make_muon_config(64, 64, coefficients=coef, steps=12)
    h = ctypes.c_void_p()
    st = lib.mlpb_muon_create(ctypes.byref(cfg), ctypes.byref(h))
    assert st in (mlpb.MLPB_OK, mlpb.MLPB_ECUDA)
    lib.mlpb_muon_destroy(h)


def test_null_arguments(lib):
    E, n = mlpb.MLPB_EINVAL, ctypes.c_size_t()
    assert lib.mlpb_muon_create(None, None) == E
    assert lib.mlpb_muon_workspace_size(None, ctypes.byref(n)) == E
    assert lib.mlpb_muon_orthogonalize(None, 1, 0, 1, 1, None) == E
    assert lib.mlpb_muon_step(None, *[None] * 7) == E
    assert lib.mlpb_muon_last_device_error(None, None) == E
    lib.mlpb_muon_destroy(None)


def test_header_flag_values_match_binding():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                            "include", "mlpb.h")).read()
    m = re.search(r"#define\s+MLPB_MUON_FAULT_INJECT\s+(0x[0-9a-fA-F]+)u", src)
    assert m and int(m.group(1), 16) == mlpb.MLPB_MUON_FAULT_INJECT
