"""A projection as it is trained and served: the weight laid out in block-scaled E4M3, forward,
backward over two micro-batches, the orthogonalised update, and the updated weight laid out again;
and the update of the MLP block's own weight gradients.  Every stage is compared with the fp64
oracles from the inputs that the stage before it left on the GPU."""
import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from oracle import b128, muon

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _randn(seed, *shape, std=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _update_close(W, W0, M0, G, plan, lr):
    """W after a step from W0, M0 and G (all [r][c])."""
    c = plan.cfg
    want, _, O, U = muon.step(W0, M0, G, lr, c.momentum, bool(c.nesterov), c.weight_decay, c.scale)
    moved = np.linalg.norm(muon.rounded(U) - O) + 1e-6 * np.linalg.norm(O)
    d = np.maximum(np.abs(W - want) - 2.0 ** -21 * np.abs(W0), 0)
    assert np.linalg.norm(d) <= 3 * lr * c.scale * moved


@pytest.mark.parametrize("T,K,N", [(70, 264, 200), (24, 136, 520)])
def test_two_steps_of_a_projection(T, K, N):
    layer = mlpb.Linear8(T, K, N)
    serving = mlpb.Linear8(4, K, N, training=False)
    update = mlpb.Muon(N, K, momentum=0.9, weight_decay=0.1, scale=0.2 * max(N, K) ** 0.5)
    W, M = _randn(1, N, K, std=K ** -0.5), torch.zeros(N, K, device="cuda")
    Wb = torch.empty(N, K, dtype=BF, device="cuda")
    lr = torch.tensor([0.02], device="cuda")
    rate = float(np.float32(0.02))
    layer.load(W)
    for step in range(2):
        dW = torch.zeros(N, K, device="cuda")
        want = np.zeros((N, K))
        mags = np.zeros((N, K))
        w_now = _np(W if step == 0 else Wb)
        for micro in range(2):
            X = _randn(10 * step + micro, T, K, dtype=BF)
            dY = _randn(10 * step + micro + 5, T, N, std=1e-2, dtype=BF)
            Y = layer.forward(X)
            dX, _ = layer.backward(dY, dW=dW, accumulate=True)
            o = b128.linear(_np(X), w_now, _np(dY))
            for got, k, terms in ((Y, "Y", K), (dX, "dX", N)):
                tol = (terms / 32 + 4) * 2.0 ** -22 * o[k][1] + 2.0 ** -8 * np.abs(o[k][0])
                assert (np.abs(_np(got) - o[k][0]) <= tol).all(), k
            want += o["dW"][0]
            mags += o["dW"][1]
        assert (np.abs(_np(dW) - want) <= (T / 32 + 6) * 2.0 ** -22 * mags).all()
        before = _np(W), _np(M)
        update.step(W, M, dW, lr, Wb=Wb)
        _update_close(_np(W), *before, _np(dW), update, rate)
        assert torch.equal(Wb, W.to(BF))
        layer.load(Wb)
    serving.load(Wb)
    X = _randn(99, 3, K, dtype=BF)
    assert torch.equal(serving.forward(X), layer.forward(X))
    assert mlpb.mlpb_linear8_last_device_error(layer.handle) == mlpb.MLPB_OK
    assert mlpb.mlpb_muon_last_device_error(update.handle) == mlpb.MLPB_OK


def test_update_of_the_blocks_gradients():
    """dW1 [t][2][Fs][H] and dW2 [t][H][Fs] of a SwiGLU block, each shard's matrices by themselves."""
    T, H, F, t = 128, 192, 256, 2
    blk = mlpb.MLPBlock(T, H, F, t, "swiglu", has_bias=False)
    W1 = _randn(1, t, 2, F // t, H, std=H ** -0.5, dtype=BF)
    W2 = _randn(2, t, H, F // t, std=F ** -0.5, dtype=BF)
    blk.forward(_randn(3, T, H, dtype=BF), W1, None, W2, None)
    grads = blk.backward(_randn(3, T, H, dtype=BF), W1, W2, _randn(4, T, H, std=1e-2, dtype=BF))
    for W, G in ((W1, grads["dW1"]), (W2, grads["dW2"])):
        r, c = W.shape[-2:]
        plan = mlpb.Muon(r, c, W.numel() // (r * c), scale=0.2 * max(r, c) ** 0.5)
        master, M = W.float(), torch.zeros_like(G)
        before = _np(master).reshape(-1, r, c)
        lr = torch.tensor([0.01], device="cuda")
        plan.step(master, M, G, lr, Wb=W)  # the block's bf16 weight is the copy
        assert torch.equal(W, master.to(BF)) and torch.equal(M, G)
        after, g = _np(master).reshape(-1, r, c), _np(G).reshape(-1, r, c)
        for i in range(len(after)):
            _update_close(after[i], before[i], np.zeros((r, c)), g[i], plan,
                          float(np.float32(0.01)))
    blk.close()


def test_a_step_in_a_graph():
    """Layout, forward, backward and update captured together and replayed twice from the same
    state: the same bits as eager calls."""
    T, K, N = 40, 200, 136
    X, dY = _randn(1, T, K, dtype=BF), _randn(2, T, N, std=1e-2, dtype=BF)
    W0, M0 = _randn(3, N, K, std=0.05), _randn(4, N, K, std=1e-2)
    lr = torch.tensor([0.05], device="cuda")
    layer, update = mlpb.Linear8(T, K, N), mlpb.Muon(N, K)
    W, M = W0.clone(), M0.clone()
    Y, dX = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, K, dtype=BF, device="cuda")
    dW = torch.empty(N, K, device="cuda")

    def step():
        layer.load(W)
        layer.forward(X, Y=Y)
        layer.backward(dY, dX=dX, dW=dW)
        update.step(W, M, dW, lr)
    step()
    step()
    want = [t.clone() for t in (W, M, Y, dX, dW)]
    W.copy_(W0)
    M.copy_(M0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    W.copy_(W0)
    M.copy_(M0)
    graph.replay()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((W, M, Y, dX, dW), want))
