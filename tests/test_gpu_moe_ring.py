"""The mixture-of-experts kernel's rings under long sums: a stage that is refilled while a warp still
reads it gives single wrong outputs now and then, at other places in every call.  So every call is
held to the first one's bits (sums run in a fixed order), and the first to 64 bits.

Bound of the parity check, for the routing that the call returned (u = 2^-24; a tensor-core sum
counts 2 u a step of 16): pre-activations are within (H / 16 + 32) 2 u of sum |x||w|; act' is at
most 1.13; a is rounded to bf16 (2^-8 with its sigmoid's 4e-5); Y adds (K F / 16 + 32) 2 u of its
magnitude and half a bf16 step.
"""
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16


def _make(T, H, F, E, seed=0):
    g = torch.Generator(device="cuda").manual_seed(T * 10000 + H + F + E + seed)

    def n(*shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)
    return (n(T, H, std=1.0), n(E, H, std=H ** -0.5), n(E, 2, F, H, std=H ** -0.5),
            n(E, H, F, std=F ** -0.5))


def _parity(d, K, out):
    """|Y - ref| over its bound, at most."""
    X, Wr, W1, W2 = d
    Y, ids, w = out
    T, H = X.shape
    F = W2.shape[2]
    x = X.double()
    ref, bound = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(2))
    pre, post = (H / 16 + 32) * 2 * U, (K * F / 16 + 32) * 2 * U
    for e in range(W2.shape[0]):
        m = (w * (ids == e)).sum(1).double()[:, None]
        if not (m != 0).any():
            continue
        (g, u), (g_err, u_err) = ([x @ W1[e, i].double().T for i in range(2)],
                                  [pre * (x.abs() @ W1[e, i].double().abs().T) for i in range(2)])
        a = g * torch.sigmoid(g) * u
        silu = g.abs() * torch.sigmoid(g.abs())  # >= |silu(g)|
        a_err = 1.13 * u.abs() * g_err + silu * u_err + 4e-5 * a.abs()
        a_err = a_err + 2.0 ** -8 * (a.abs() + a_err)
        w2 = W2[e].double()
        ref += m * (a @ w2.T)
        bound += m * ((a_err + post * a.abs()) @ w2.abs().T)
    bound += 2.0 ** -8 * (ref.abs() + bound) + 1e-30
    return ((Y.double() - ref).abs() / bound).max().item()


# (tokens, hidden, ffn, experts, topk): fc2 in 33 steps of K whose last holds 8 columns, with one
# token tile, two (three stages a ring), and more than 16 tokens of an expert (one ring for the
# CTA); several units a group; a sum of one step; GELU-width units are the other tests'
@pytest.mark.parametrize("T,H,F,E,K", [(3, 4096, 8200, 3, 3), (12, 4096, 8200, 2, 2),
                                       (16, 2048, 4104, 3, 3), (40, 4096, 8200, 2, 2),
                                       (64, 2048, 2056, 4, 3), (1, 8192, 1032, 16, 8),
                                       (9, 256, 256, 8, 4)])
def test_every_call_has_the_first_ones_bits(T, H, F, E, K):
    d = _make(T, H, F, E)
    plan = mlpb.MoEDecode(T, H, F, E, K)
    first = plan.forward(*d)
    assert mlpb.mlpb_moe_last_device_error(plan.handle) == 0
    assert _parity(d, K, first) <= 1
    out = [torch.empty_like(t) for t in first]
    busy = torch.zeros(16 << 20, device="cuda")
    wrong = torch.zeros(3, dtype=torch.int64, device="cuda")  # values, over all calls
    for i in range(400):
        if i % 3 == 0:
            busy.add_(1)  # the weights leave L2 now and then
        plan.forward(*d, *out)
        wrong += torch.stack([(a != b).sum() for a, b in zip(out, first)])
    assert mlpb.mlpb_moe_last_device_error(plan.handle) == 0
    assert wrong.tolist() == [0, 0, 0]
