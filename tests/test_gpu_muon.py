"""The orthogonalised update against the fp64 oracle (oracle/muon.py).

Tolerances.  The polynomial steps amplify roundings differently for each input, so the oracle says
for each one how far the fp16 operands move its result (the same steps in 64 bits with these
operands rounded); the library, whose sums are fp32 besides, may be three times as far, in the
2-norm over a matrix, and the bf16 result is off by half a step more, 2^-8 of each value.  A single
element may be off by six times the largest error of those roundings.  (Six: 30 times an element's
share of the norm, which is 4.7 shares at most for even matrices; where rows differ in size the
roundings' own largest error is some 100 shares, since each is relative to its element.)  M is one
fused fp32 multiplication and addition: one rounding of a product and a sum, 2^-23 of their
magnitudes."""
import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from oracle import muon

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _randn(seed, *shape, std=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _close(got, U, half=True, steps=5, coef=muon.COEF, scale=1.0, more=0.0):
    """got [n][r][c] is `scale` times the orthogonalisation of U [n][r][c]."""
    for g, u in zip(_np(got), U):
        want = muon.orthogonalize(u, steps, coef)
        e = muon.rounded(u, steps, coef) - want
        moved = np.linalg.norm(e) + 1e-6 * np.linalg.norm(want)
        d = np.abs(g / scale - want)
        d = np.maximum(d - (2.0 ** -8 * np.abs(want) if half else 0.0) - more / scale, 0.0)
        assert np.linalg.norm(d) <= 3 * moved, (np.linalg.norm(d), moved)
        assert d.max() <= 6 * (np.abs(e).max() + 1e-6 * np.abs(want).max()), (d.max(), moved)


SHAPES = [(1, 1, 1), (1, 1, 40), (2, 40, 1), (1, 16, 16), (3, 33, 77), (2, 130, 65), (1, 64, 1032),
          (1, 300, 257), (2, 257, 600), (1, 520, 264), (1, 128, 256), (5, 96, 128), (1, 700, 700),
          # in shared memory: sides around 32 and 128, one CTA and clusters, long sides that no
          # longer fit
          (1, 32, 2000), (3, 2001, 31), (1, 97, 1000), (2, 128, 4096), (1, 4100, 128), (40, 20, 70),
          (1, 127, 4097), (1, 9000, 60), (200, 8, 8), (1, 24, 8300)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,r,c", SHAPES)
def test_orthogonalize(n, r, c, dtype):
    U = _randn(r * c, n, r, c, std=1e-3, dtype=dtype)
    plan = mlpb.Muon(r, c, n)
    plan.workspace.fill_(0xff)  # NaN: nothing is read that was not written
    O = plan.orthogonalize(U)
    assert mlpb.mlpb_muon_last_device_error(plan.handle) == mlpb.MLPB_OK
    _close(O, _np(U))
    assert torch.equal(plan.orthogonalize(U), O)  # the same bits


@pytest.mark.parametrize("r,c", [(200, 333), (333, 200), (64, 512)])
@pytest.mark.parametrize("kind", ["low_rank", "decaying", "rank_one", "wide_range"])
def test_spectra(kind, r, c):
    k = min(r, c)
    a, b = _randn(1, r, k), _randn(2, k, c)
    if kind == "low_rank":
        U = a[:, :8] @ b[:8] + 0.05 * _randn(3, r, c)
    elif kind == "decaying":
        U = (a / torch.arange(1, k + 1, device="cuda")) @ b
    elif kind == "rank_one":
        U = a[:, :1] @ b[:1]
    else:
        U = _randn(4, r, c) * torch.exp(3 * _randn(5, r, 1)) * torch.exp(2 * _randn(6, 1, c))
    O = mlpb.Muon(r, c).orthogonalize(U[None])
    _close(O, _np(U[None]))


@pytest.mark.parametrize("steps,coef", [(1, muon.COEF), (2, muon.COEF), (6, muon.COEF),
                                        (10, (1.5, -0.5, 0.0)), (8, (1.875, -1.25, 0.375))])
@pytest.mark.parametrize("r,c", [(72, 200), (200, 72)])
def test_steps_and_coefficients(r, c, steps, coef):
    U = _randn(7, 2, r, c)
    O = mlpb.Muon(r, c, 2, steps=steps, coefficients=coef).orthogonalize(U)
    _close(O, _np(U), steps=steps, coef=tuple(float(np.float32(x)) for x in coef))


def test_sizes_near_the_ends_of_fp32():
    U = _randn(1, 40, 56)
    plan = mlpb.Muon(40, 56)
    want = plan.orthogonalize(U)
    for f in (2.0 ** -120, 2.0 ** -60, 2.0 ** 60, 2.0 ** 120):
        assert torch.equal(plan.orthogonalize(U * f), want)  # powers of two: the same bits
    tiny = torch.full((40, 56), 2.0 ** -149, device="cuda")
    _close(plan.orthogonalize(tiny)[None], _np(tiny)[None])
    mixed = U.clone()
    mixed[:, 0] *= 2.0 ** 60
    mixed[:, 1] *= 2.0 ** -60
    _close(plan.orthogonalize(mixed)[None], _np(mixed)[None])


def test_zero_infinite_and_nan_matrices_keep_to_themselves():
    U = _randn(1, 6, 48, 70)
    plan = mlpb.Muon(48, 70, 6)
    want = plan.orthogonalize(U)
    hurt = U.clone()
    hurt[0] = 0
    hurt[2, 5, 7] = float("inf")
    hurt[3, 0, 0] = float("nan")
    O = plan.orthogonalize(hurt)
    assert not bool(O[0].any())
    assert bool(O[2:4].isnan().all())
    for i in (1, 4, 5):
        assert torch.equal(O[i], want[i])


@pytest.mark.parametrize("shape", [(2, 2, 40, 72), (3, 130, 48), (1, 77, 33), (2, 200, 264),
                                   (1, 333, 141)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_step(shape, nesterov):
    n, (r, c) = int(np.prod(shape[:-2])), shape[-2:]
    mu, decay, scale, lr = 0.9, 0.1, 0.2 * max(r, c) ** 0.5, 0.05
    W, M, G = _randn(1, *shape, std=0.05), _randn(2, *shape, std=1e-2), _randn(3, *shape, std=1e-2)
    plan = mlpb.Muon(r, c, n, momentum=mu, nesterov=nesterov, weight_decay=decay, scale=scale)
    w, m, wb = W.clone(), M.clone(), torch.empty(shape, dtype=BF, device="cuda")
    rate = torch.tensor([lr], device="cuda")
    plan.step(w, m, G, rate, Wb=wb)
    flat = [_np(t).reshape(n, r, c) for t in (W, M, G, w, m)]
    mu32, lr32 = float(np.float32(mu)), float(np.float32(lr))
    decay32, scale32 = float(np.float32(decay)), float(np.float32(scale))
    for W0, M0, G0, w0, m0 in zip(*flat):
        want_w, want_m, O, U = muon.step(W0, M0, G0, lr32, mu32, nesterov, decay32, scale32)
        assert (np.abs(m0 - want_m) <= 2.0 ** -23 * (np.abs(mu32 * M0) + np.abs(G0))).all()
        moved = np.linalg.norm(muon.rounded(U) - O) + 1e-6 * np.linalg.norm(O)
        d = np.abs(w0 - want_w) - 2.0 ** -21 * np.abs(W0)
        assert np.linalg.norm(np.maximum(d, 0)) <= 3 * lr * scale * moved
    assert torch.equal(wb, w.to(BF))
    again_w, again_m = W.clone(), M.clone()
    plan.step(again_w, again_m, G, rate)  # without the copy
    assert torch.equal(again_w, w) and torch.equal(again_m, m)
    O = plan.orthogonalize(_randn(9, *shape))  # the plan's other call, its shape kept
    assert O.shape == shape


def test_graph_streams_and_two_plans():
    r, c = 96, 130
    U = _randn(1, 2, r, c)
    plan = mlpb.Muon(r, c, 2)
    want = plan.orthogonalize(U)
    x, o = torch.zeros_like(U), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.orthogonalize(x, o)
    x.copy_(U)
    for _ in range(2):
        graph.replay()
        assert torch.equal(o, want)
    side, other = torch.cuda.Stream(), mlpb.Muon(r, c, 2)
    torch.cuda.synchronize()
    a = other.orthogonalize(U, stream=side)
    b = plan.orthogonalize(U)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_refusals():
    plan = mlpb.Muon(24, 40, 2)
    U = _randn(1, 2, 24, 40)
    lr = torch.ones(1, device="cuda")
    with pytest.raises(ValueError, match="matrices"):
        plan.orthogonalize(U[:1])
    with pytest.raises(ValueError, match="matrices"):
        plan.orthogonalize(U.transpose(1, 2).contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        plan.orthogonalize(_randn(1, 2, 40, 24).transpose(1, 2))
    with pytest.raises(TypeError):
        plan.orthogonalize(U.half())
    with pytest.raises(ValueError, match="are needed"):
        mlpb.mlpb_muon_orthogonalize(plan.handle, U, torch.empty_like(U, dtype=BF),
                                     plan.workspace[:64])
    with pytest.raises(mlpb.MLPBError):
        mlpb.mlpb_muon_orthogonalize(plan.handle, U, None, plan.workspace)
    with pytest.raises(TypeError):
        plan.step(U.clone(), U.clone(), U.to(BF), lr)
    with pytest.raises(ValueError, match="CUDA"):
        plan.step(U.clone(), U.clone(), U, torch.ones(1))
    with pytest.raises(mlpb.MLPBError):
        plan.step(U.clone(), U.clone(), U, None)


def test_an_expired_wait_is_reported_and_the_next_call_is_right():
    U = _randn(1, 1, 300, 520)  # no matrix of shared memory: nothing waits for a copy there
    want = mlpb.Muon(300, 520).orthogonalize(U)
    hurt = mlpb.Muon(300, 520, flags=mlpb.MLPB_MUON_FAULT_INJECT)
    hurt.orthogonalize(U)
    assert mlpb.mlpb_muon_last_device_error(hurt.handle) == mlpb.MLPB_ETIMEOUT
    assert torch.equal(hurt.orthogonalize(U), want)
    assert mlpb.mlpb_muon_last_device_error(hurt.handle) == mlpb.MLPB_OK


@pytest.mark.parametrize("n,r,c", [(32, 4096, 64), (32, 64, 4096), (16, 128, 2000)])
def test_the_form_goes_by_the_steps_too(n, r, c):
    """Matrices that a cluster's shared memory holds, and that the tiled products finish sooner
    where there are few steps: either form against the oracle."""
    U = _randn(r, n, r, c)
    small = []
    for steps, coef in ((1, muon.COEF), (3, muon.COEF), (12, (1.5, -0.5, 0.0))):
        plan = mlpb.Muon(r, c, n, steps=steps, coefficients=coef)
        small.append(plan.workspace.numel() == 256)
        O = plan.orthogonalize(U)
        assert mlpb.mlpb_muon_last_device_error(plan.handle) == mlpb.MLPB_OK
        _close(O[:3], _np(U[:3]), steps=steps, coef=coef)
        _close(O[-1:], _np(U[-1:]), steps=steps, coef=coef)
    assert small == sorted(small) and small[-1]  # once it pays, it pays with more steps


def _spectrum(kind, r, c, seed):
    g = np.random.default_rng(seed)
    k = min(r, c)
    a, b = g.standard_normal((r, k)), g.standard_normal((k, c))
    if kind == "gaussian":
        return g.standard_normal((r, c))
    if kind == "gradient":  # strong directions that fall off, and noise
        m = max(1, k // 16)
        return (a[:, :m] / m ** 0.5) @ (b[:m] * np.logspace(0, -1.5, m)[:, None]) \
            + 0.2 * g.standard_normal((r, c))
    if kind == "low_rank":
        return a[:, :8] @ b[:8] + 0.05 * g.standard_normal((r, c))
    if kind == "decaying":
        return (a / np.arange(1, k + 1)) @ b
    if kind == "decaying far":
        return (a * np.logspace(0, -4, k)) @ b
    return a[:, :1] @ b[:1] + (1e-3 * g.standard_normal((r, c)) if kind == "one and noise" else 0)


# Errors in the 2-norm, of O's.  The roundings of the operands alone, in 64 bits (oracle/muon.py),
# reach three quarters of these over eight seeds at the sizes below (n = 16: 2.6e-3 at most); what
# the library's fp32 sums add is some 1e-6.
SPECTRA = {"gaussian": 1e-3, "gradient": 1e-3, "low_rank": 1e-3, "decaying": 1.2e-3,
           "decaying far": 1.8e-3, "one": 3e-3, "one and noise": 2.4e-3}


@pytest.mark.parametrize("kind", SPECTRA)
@pytest.mark.parametrize("r,c", [(64, 512), (200, 333), (333, 200), (1024, 32), (16, 64)])
def test_errors_of_each_spectrum(r, c, kind):
    """O in fp32 (a step from a zero weight) against bounds that do not move with the format."""
    U = np.float32(_spectrum(kind, r, c, r + c))
    plan = mlpb.Muon(r, c, momentum=0.0, scale=-1.0)
    W, M = (torch.zeros(r, c, device="cuda") for _ in range(2))
    plan.step(W, M, torch.from_numpy(U).cuda(), torch.ones(1, device="cuda"))
    want = muon.orthogonalize(U)
    e = np.linalg.norm(_np(W) - want) / np.linalg.norm(want)
    assert e <= (3.5e-3 if min(r, c) < 32 else SPECTRA[kind]), e


@pytest.mark.parametrize("r,c", [(64, 512), (333, 200), (500, 700)])
@pytest.mark.parametrize("kind", ["gaussian", "decaying far", "one and noise"])
def test_errors_of_many_steps(r, c, kind):
    """12 steps: roundings amplified 3.4 times a step come up only where U holds nothing (the
    operands' roundings: 3e-3 of O at most)."""
    U = np.float32(_spectrum(kind, r, c, r + c))
    plan = mlpb.Muon(r, c, momentum=0.0, scale=-1.0, steps=12)
    W, M = (torch.zeros(r, c, device="cuda") for _ in range(2))
    plan.step(W, M, torch.from_numpy(U).cuda(), torch.ones(1, device="cuda"))
    want = muon.orthogonalize(U, 12)
    assert np.linalg.norm(_np(W) - want) <= 5e-3 * np.linalg.norm(want)


@pytest.mark.parametrize("n,r,c", [(1, 1, 65536), (1, 65536, 1), (65535, 1, 3), (65535, 2, 1),
                                   (1, 16, 65536), (1, 65536, 40), (1, 65535, 129)])
def test_longest_sides_and_most_matrices(n, r, c):
    U = _randn(r + c, n, r, c)
    plan = mlpb.Muon(r, c, n)
    plan.workspace.fill_(0xff)
    O = plan.orthogonalize(U)
    assert mlpb.mlpb_muon_last_device_error(plan.handle) == mlpb.MLPB_OK
    pick = sorted({0, n // 2, n - 1})
    _close(O[pick], _np(U[pick]))
    assert bool(O.isfinite().all()) and bool((O != 0).flatten(1).any(1).all())
