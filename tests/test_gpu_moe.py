"""GPU parity of the mixture-of-experts MLP for a few tokens against its fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24; a tensor-core sum is counted at 2 u a step, K / 16
steps).  Logits are fp32 sums of at most 8 ceil(H / 4096) + 5 + 16 roundings: within D =
(8 ceil(H / 4096) + 24) u of their magnitude sum |x||wr|.  An id must be the oracle's where the
logits before and after it in the order are further away than 2 D; the weights are within 2 D + 16 u, twice that when normalised.  Pre-activations are within
(H / 16 + 32) 2 u of sum |x||w|; act' is at most 1.13; a is rounded to bf16 (2^-8 with its
sigmoid's 4e-5); Y adds (pairs' K / 16 + 32) 2 u of its magnitude and half a bf16 step.
"""
import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from oracle import moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16

# (tokens, hidden, ffn, experts, topk): one of everything, widths under a step of K and not
# whole steps of it, tokens at the borders of the tiles of eight, experts with more than 32
# tokens, every expert taken, the most experts and choices
SHAPES = [(1, 8, 8, 1, 1), (1, 64, 8, 2, 1), (1, 4096, 1376, 16, 8), (3, 72, 40, 5, 3),
          (7, 328, 200, 16, 2), (8, 256, 64, 4, 4), (9, 512, 136, 12, 2), (16, 320, 104, 12, 4),
          (17, 1000, 136, 7, 2), (32, 264, 72, 32, 8), (33, 512, 64, 3, 2), (40, 1288, 56, 1, 1),
          (64, 2048, 264, 8, 2), (64, 512, 64, 256, 16), (5, 4104, 48, 200, 16)]


def _make(T, H, F, E, act, seed=0):
    g = torch.Generator().manual_seed(T * 10000 + H + F + E + seed)

    def n(*shape, std):
        return (torch.randn(shape, generator=g) * std).to(BF)
    w1 = (E, 2, F, H) if act == "swiglu" else (E, F, H)
    return (n(T, H, std=1.0), n(E, H, std=H ** -0.5), n(*w1, std=H ** -0.5),
            n(E, H, F, std=F ** -0.5))


def _check(d, K, act, norm, out):
    X, Wr, W1, W2 = (t.double().numpy() for t in d)
    Y, ids, w = (t.double().cpu().numpy() for t in out)
    ids = ids.astype(int)
    T, H = X.shape
    E, F = W2.shape[0], W2.shape[2]
    l, ids_ref, _ = moe.route(X, Wr, K, norm)
    D = (8 * -(-H // 4096) + 24) * U * (np.abs(X) @ np.abs(Wr).T).max(1)
    # a place in the order is settled where the logits beside it are further away than 2 D
    s = -np.sort(-l, axis=1)[:, :K + 1]
    apart = np.ones((T, K + 1), bool)
    apart[:, 1:s.shape[1]] = s[:, :-1] - s[:, 1:] > 2 * D[:, None]
    settled = apart[:, :K] & apart[:, 1:]
    assert settled.mean() >= 0.9
    assert np.array_equal(ids[settled], ids_ref[settled])
    assert all(len(set(row)) == K for row in ids.tolist())
    p = np.exp(l - l.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w_ref = np.take_along_axis(p, ids, 1)
    if norm:
        w_ref = w_ref / w_ref.sum(1, keepdims=True)
    rel = (2 * D + 16 * U) * (2 if norm else 1)
    assert (np.abs(w - w_ref) <= rel[:, None] * w_ref + 1e-37).all()
    ref = moe.forward(X, W1, W2, ids, w_ref, act)
    bound, spread = np.zeros_like(ref), 0.0
    pre, post = (H / 16 + 32) * 2 * U, (K * F / 16 + 32) * 2 * U
    for t in range(T):
        for k, e in enumerate(ids[t]):
            a, z = moe.activation(X[t], W1[e], act)
            z_err = pre * (np.abs(W1[e]) @ np.abs(X[t]))
            if act == "gelu":
                a_err = 1.13 * z_err + 4e-5 * np.abs(a)
            else:
                g, u = z
                sg = np.abs(g) / (1 + np.exp(-np.abs(g)))  # >= |silu(g)|
                a_err = 1.13 * np.abs(u) * z_err[0] + sg * z_err[1] + 4e-5 * np.abs(a)
            a_err = a_err + (2.0 ** -8 + rel[t]) * (np.abs(a) + a_err)
            m = w_ref[t, k] * np.abs(W2[e])
            bound[t] += m @ a_err + post * (m @ np.abs(a))
            spread += ((m * a) ** 2).sum()
    bound += 2.0 ** -8 * (np.abs(ref) + bound) + 1e-30
    assert (np.abs(Y - ref) <= bound).all(), float((np.abs(Y - ref) / bound).max())
    # That bound is of the worst case.  The roundings of a are independent, each within 2^-8 |a|,
    # so their sum in an output has a variance of at most a third of 2^-16 sum (w W2 a)^2 (a
    # third: uniform within the half step); without the third it is three times what is due.
    assert np.linalg.norm(Y - ref) <= 2.0 ** -8 * np.sqrt(spread + (ref ** 2).sum())


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("T,H,F,E,K", SHAPES)
def test_forward(T, H, F, E, K, act):
    d = _make(T, H, F, E, act)
    norm = act == "swiglu"
    plan = mlpb.MoEDecode(T, H, F, E, K, act, norm)
    out = plan.forward(*(t.cuda() for t in d))
    torch.cuda.synchronize()
    assert mlpb.mlpb_moe_last_device_error(plan.handle) == 0
    _check(d, K, act, norm, out)


def test_fewer_tokens_than_the_handle_admits():
    """One handle serves calls of any number of tokens, one after the other, and writes no row
    beyond them."""
    d = _make(64, 520, 72, 12, "swiglu")
    plan = mlpb.MoEDecode(64, 520, 72, 12, 3)
    g = [t.cuda() for t in d]
    full = plan.forward(*g)
    for T in (1, 0, 30, 8, 64):
        Y = torch.full((64, 520), 5.0, dtype=BF, device="cuda")
        ids = torch.full((64, 3), -7, dtype=torch.int32, device="cuda")
        w = torch.full((64, 3), 9.0, device="cuda")
        plan.forward(g[0][:T], *g[1:], Y=Y[:T], ids=ids[:T], weights=w[:T])
        torch.cuda.synchronize()
        assert torch.equal(ids[:T], full[1][:T]) and torch.equal(w[:T], full[2][:T])
        _check((d[0][:T], *d[1:]), 3, "swiglu", True, (Y[:T], ids[:T], w[:T])) if T else None
        assert (Y[T:] == 5).all() and (ids[T:] == -7).all() and (w[T:] == 9).all()
    assert mlpb.mlpb_moe_last_device_error(plan.handle) == 0


def test_equal_logits_take_the_lowest_index():
    d = list(_make(6, 264, 40, 10, "swiglu"))
    d[1] = d[1][:1].expand(10, -1).contiguous()      # ten equal router rows
    plan = mlpb.MoEDecode(6, 264, 40, 10, 4)
    Y, ids, w = plan.forward(*(t.cuda() for t in d))
    assert (ids.cpu() == torch.arange(4, dtype=torch.int32)).all()
    assert (w == 0.25).all()
    _, ids, _ = plan.forward(torch.zeros_like(d[0]).cuda(), *(t.cuda() for t in d[1:]))
    assert (ids.cpu() == torch.arange(4, dtype=torch.int32)).all()


def test_bad_tokens_stay_alone():
    """A token of NaN and one of infinities choose valid experts and spoil no other token."""
    d = _make(12, 264, 40, 10, "gelu")
    plan = mlpb.MoEDecode(12, 264, 40, 10, 3, "gelu")
    good = plan.forward(*(t.cuda() for t in d))
    X = d[0].clone()
    X[2], X[7, 5] = float("nan"), float("inf")
    Y, ids, w = plan.forward(X.cuda(), *(t.cuda() for t in d[1:]))
    assert ((ids >= 0) & (ids < 10)).all()
    assert torch.isnan(Y[2]).all()
    for t in (2, 7):
        assert len(set(ids[t].tolist())) == 3
    keep = [t for t in range(12) if t not in (2, 7)]
    for a, b in zip(good, (Y, ids, w)):
        assert torch.equal(a[keep], b[keep])


def test_same_bits_stream_and_two_graphs():
    d = [t.cuda() for t in _make(20, 1032, 136, 16, "swiglu")]
    plan = mlpb.MoEDecode(20, 1032, 136, 16, 4)
    want = plan.forward(*d)
    for a, b in zip(want, plan.forward(*d)):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = plan.forward(*d)
    s.synchronize()
    assert torch.equal(got[0], want[0])
    graphs = []
    for _ in range(2):
        p2 = mlpb.MoEDecode(20, 1032, 136, 16, 4)
        out = p2.forward(*d)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            p2.forward(*d, *out)
        for t in out:
            t.zero_()
        graphs.append((gr, out, p2))
    for _ in range(3):
        for gr, *_ in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for _, out, p2 in graphs:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert mlpb.mlpb_moe_last_device_error(p2.handle) == 0


@pytest.mark.parametrize("T,F", [(17, 40), (24, 264), (33, 72), (41, 256), (55, 520), (64, 1032)])
def test_tokens_of_an_expert(T, F):
    """Every number of token tiles for one expert next to experts with few or none: a router that
    sends all tokens to expert 1, and their second choice where it falls; several units a CTA."""
    for H, act in ((264, "gelu"), (4104, "swiglu")):
        d = list(_make(T, H, F, 9, act))
        d[0][:, 0] = 8.0
        d[1][1, 0] = 2.0
        plan = mlpb.MoEDecode(64, H, F, 9, 2, act)
        g = [t.cuda() for t in d]
        out = plan.forward(*g)
        assert (out[1][:, 0] == 1).sum() >= T - 1
        _check(d, 2, act, True, out)
        again = plan.forward(*g)
        assert all(torch.equal(a, b) for a, b in zip(out, again))
        assert mlpb.mlpb_moe_last_device_error(plan.handle) == 0


def test_two_handles_at_once_and_forms_in_turn():
    """Handles on two streams at the same time; one handle with calls of a few and of many tokens
    an expert after each other; a call after another one left NaN in shared memory."""
    d = [t.cuda() for t in _make(64, 1024, 520, 6, "swiglu")]
    xs, hs = (d[0], d[0][:1].contiguous()), [mlpb.MoEDecode(64, 1024, 520, 6, 2) for _ in range(2)]
    want = [[t.clone() for t in h.forward(x, *d[1:])] for h, x in zip(hs, xs)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in hs], [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(hs[i].forward(xs[i], *d[1:]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for o in outs[i] for a, b in zip(o, want[i]))
    for T in (1, 64, 5, 40, 17, 2, 33):
        x = d[0][:T].contiguous()
        fresh = mlpb.MoEDecode(64, 1024, 520, 6, 2).forward(x, *d[1:])
        assert all(torch.equal(a, b) for a, b in zip(hs[0].forward(x, *d[1:]), fresh))
    odd = [t.cuda() for t in _make(64, 1000, 264, 4, "swiglu")]
    plan = mlpb.MoEDecode(64, 1000, 264, 4, 2)
    a = [t.clone() for t in plan.forward(*odd)]
    hs[1].forward(torch.full_like(d[0], float("nan")), *d[1:])
    assert all(torch.equal(u, v) for u, v in zip(a, plan.forward(*odd)))
    for h in (*hs, plan):
        assert mlpb.mlpb_moe_last_device_error(h.handle) == 0


def test_offsets_past_32_bits():
    """Weights of more than 2^32 elements: the last experts are those of a small layer with the
    same rows (the first ones, of zeros, have logits of zero and are not taken)."""
    T, H, F, E, n = 3, 4096, 8200, 66, 3
    d = [t.cuda() for t in _make(T, H, F, n, "swiglu")]
    d[1] = (d[0][:1].float().sign() * d[1].float().abs() + 0.0).to(BF)  # token 0 takes them
    d[0] = d[0][:1].expand(T, -1).contiguous()
    Wr = torch.zeros(E, H, dtype=BF, device="cuda")
    W1 = torch.zeros(E, 2, F, H, dtype=BF, device="cuda")
    W2 = torch.zeros(E, H, F, dtype=BF, device="cuda")
    Wr[-n:], W1[-n:], W2[-n:] = d[1], d[2], d[3]
    big, small = mlpb.MoEDecode(T, H, F, E, n), mlpb.MoEDecode(T, H, F, n, n)
    Y, ids, w = big.forward(d[0], Wr, W1, W2)
    y, ids2, w2 = small.forward(*d)
    assert torch.equal(ids, ids2 + (E - n))
    # The two sum their logits in different orders (the first form of this test held them equal
    # to 2^-20, which forgets that): each is within D of the exact ones, its normalised weights
    # within 2 (2 D + 16 u), the two within twice that of each other.
    x = d[0][0].double()
    D = (8 * -(-H // 4096) + 24) * U * (d[1].double().abs() @ x.abs()).max().item()
    rel = 2 * 2 * (2 * D + 16 * U)
    assert ((w - w2).abs() <= rel * w2).all()
    # the outputs differ by that of the experts' weighted parts (with 1 % for their rounded
    # activations), and by a step of bf16, 2^-7 of the value
    part = torch.zeros(H, dtype=torch.float64, device="cuda")
    for k, e in enumerate(ids2[0].tolist()):
        g, u = d[2][e].double() @ x
        part += w2[0, k] * (d[3][e].double() @ (g * torch.sigmoid(g) * u)).abs()
    bound = 1.01 * rel * part + 2.0 ** -7 * y.double().abs()
    assert ((Y.double() - y.double()).abs() <= bound).all()
    assert mlpb.mlpb_moe_last_device_error(big.handle) == 0


def test_refusals():
    d = [t.cuda() for t in _make(4, 64, 32, 8, "swiglu")]
    plan = mlpb.MoEDecode(4, 64, 32, 8, 2)
    with pytest.raises(mlpb.MLPBError) as e:
        plan.forward(torch.zeros(5, 64, dtype=BF, device="cuda"), *d[1:])
    assert e.value.status == mlpb.MLPB_EUNSUPPORTED
    with pytest.raises(ValueError):
        plan.forward(d[0], d[1], d[2][:, :1].contiguous(), d[3])
    with pytest.raises(TypeError):
        plan.forward(d[0].float(), *d[1:])
    with pytest.raises(mlpb.MLPBError) as e:
        mlpb.mlpb_moe_forward(plan.handle, d[0], None, d[2], d[3], d[0].clone(),
                              torch.empty(4, 2, dtype=torch.int32, device="cuda"),
                              torch.empty(4, 2, device="cuda"), plan.workspace)
    assert e.value.status == mlpb.MLPB_EINVAL
    with pytest.raises(ValueError, match="workspace"):
        plan.workspace = plan.workspace[:256]
        plan.forward(*d)


def test_launches_in_a_row_leave_no_error():
    """The barrier's words are back at zero for the next launch, and no wait expired."""
    d = [t.cuda() for t in _make(2, 64, 32, 8, "swiglu")]
    plan = mlpb.MoEDecode(2, 64, 32, 8, 2)
    first = plan.forward(*d)
    for _ in range(50):
        out = plan.forward(*d)
    assert mlpb.mlpb_moe_last_device_error(plan.handle) == 0
    assert torch.equal(first[0], out[0])
