"""Tensors whose offsets pass 32 bits: rows, and matrices of a batch, that repeat are the same bits
wherever they lie (an element's sum does not depend on its place), and the first ones are held to
the oracles by the other tests."""
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _randn(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def test_linear_of_the_most_tokens():
    T, K, N, n = 2 ** 20, 2056, 2560, 8192  # Y has 2.7e9 elements; n rows repeat
    x, dy, W = _randn(1, n, K), _randn(2, n, N), _randn(3, N, K, std=K ** -0.5)
    small, plan = mlpb.Linear8(n, K, N), mlpb.Linear8(T, K, N)
    small.load(W)
    plan.load(W)
    y = small.forward(x)
    dx, dw = small.backward(dy)
    Y = plan.forward(x.repeat(T // n, 1))
    assert bool((Y.view(T // n, n, N) == y).all())
    del Y
    dX, dW = plan.backward(dy.repeat(T // n, 1))
    assert bool((dX.view(T // n, n, K) == dx).all())
    # codes and scales repeat, and so do the sums of each 8192 tokens (64 blocks, added in fp32):
    # 127 additions, each off by half a step of a sum of at most the whole
    assert float((dW - (T // n) * dw).abs().max()) <= 127 * 2.0 ** -24 * (T // n) \
        * float(dw.abs().max())
    assert mlpb.mlpb_linear8_last_device_error(plan.handle) == mlpb.MLPB_OK


@pytest.mark.parametrize("n,r,c", [(26000, 200, 520), (26000, 520, 200), (5200, 128, 4096),
                                   (65000, 32, 1304)])
def test_update_of_the_largest_batch(n, r, c):
    m = 4  # matrices that repeat; 2.7e9 elements
    u = _randn(1, m, r, c)
    plan = mlpb.Muon(r, c, n)
    O = plan.orthogonalize(u.repeat(n // m, 1, 1))
    assert bool((O.view(n // m, m, r, c) == O[:m]).all())
    assert bool((O[:m] != 0).any())
    want = mlpb.Muon(r, c, m).orthogonalize(u).float()
    # other tiles and ranges add in another order: some 1e-4 of an element's size, and bf16's step
    d = (O[:m].float() - want).norm() / want.norm()
    assert float(d) <= 2e-3 + 2.0 ** -8
    assert mlpb.mlpb_muon_last_device_error(plan.handle) == mlpb.MLPB_OK
