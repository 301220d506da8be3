"""The products of the block-scaled linear layer in each form that its sizes can take (results
through shared memory, from registers, in chunks; ranges of K over a cluster), against fp64 products
of what the codes stand for.  (The codes are the oracle's: test_gpu_linear8.py.)

Tolerances, as there: an MMA adds 32 exact products and cuts off at most 2^-22 of the magnitudes
added so far, so K products are off by at most (ceil(K / 32) + 4) 2^-22 of the sum of their
magnitudes.  A bf16 output adds half a step, 2^-8 of the value, an addition into what was there
2^-23 of the sum."""
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _randn(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _values(x, square=False):
    """What the codes of x stand for, fp64."""
    q = mlpb.b128_empty(*x.shape, "cuda")
    mlpb.mlpb_b128_quantize(x, q, None, square)
    return mlpb.b128_values(q, *x.shape)


def _transposed(x):
    q = mlpb.b128_empty(x.shape[1], x.shape[0], "cuda")
    mlpb.mlpb_b128_quantize(x, None, q)
    return mlpb.b128_values(q, x.shape[1], x.shape[0])


def _check(got, a, b, base=None):
    """got is a b^T (plus base) for a [m][k], b [n][k], in slices of got's columns."""
    k, step = a.shape[1], 2048
    for n0 in range(0, b.shape[0], step):
        part = b[n0:n0 + step]
        want, mags = a @ part.t(), a.abs() @ part.abs().t()
        tol = (-(-k // 32) + 4) * 2.0 ** -22 * mags
        if base is not None:
            want = want + base[:, n0:n0 + step].double()
            tol = tol + 2.0 ** -23 * want.abs()
        if got.dtype == BF:
            tol = tol + 2.0 ** -8 * want.abs()
        over = (got[:, n0:n0 + step].double() - want).abs() - tol
        bad = int((~(over <= 1e-300)).sum())
        assert bad == 0, f"{bad} from column {n0} on, {float(over.max()):.3e} over"


# More tiles than pairs of SMs, so that a pair goes from a tile at the right edge to another one; a
# 128-column half of the edge's tile holds 1 to 4 boxes (64 columns of bf16, 32 of fp32).
EDGES = [1032, 1088, 1096, 1120, 1160, 1224, 1280]


@pytest.mark.parametrize("k", [128, 200])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("edge", EDGES)
def test_short_sums_with_tiles_at_the_edge(edge, out, k):
    T = 8200
    X, W, dY = _randn(1, T, k), _randn(2, edge, k), _randn(3, T, edge)
    plan = mlpb.Linear8(T, k, edge, out_dtype=out)
    plan.load(W)
    _check(plan.forward(X), _values(X), _values(W, True))
    plan = mlpb.Linear8(T, edge, k, out_dtype=out)  # dX has the edge's width
    plan.load(W.t().contiguous())
    plan.forward(dY)
    _check(plan.backward(X)[0], _values(X), _values(W, True))
    assert mlpb.mlpb_linear8_last_device_error(plan.handle) == mlpb.MLPB_OK


@pytest.mark.parametrize("T", [100, 250, 1032])
@pytest.mark.parametrize("edge", EDGES)
def test_gradients_with_tiles_at_the_edge(edge, T):
    N = 8200
    X, dY = _randn(1, T, edge), _randn(2, T, N)
    plan = mlpb.Linear8(T, edge, N)
    plan.load(_randn(3, N, edge))
    plan.forward(X)
    a, b = _transposed(dY), _transposed(X)
    dW = plan.backward(dY, input_grad=False)[1]
    _check(dW, a, b)
    base = _randn(4, N, edge, std=T ** 0.5, dtype=F32)
    acc = base.clone()
    plan.backward(dY, dW=acc, accumulate=True, input_grad=False)
    _check(acc, a, b, base)
    assert mlpb.mlpb_linear8_last_device_error(plan.handle) == mlpb.MLPB_OK


@pytest.mark.parametrize("T", [1, 16, 300])
def test_layers_in_a_row_read_what_the_one_before_wrote(T):
    """Each launch begins while the one that writes its input ends: a chain of layers, captured and
    replayed, has the bits of one that waits for every call."""
    widths = [264, 1032, 520, 264]
    layers = []
    for i, (k, n) in enumerate(zip(widths, widths[1:])):
        layers.append(mlpb.Linear8(T, k, n))
        layers[-1].load(_randn(i, n, k, std=k ** -0.5))
    outs = [torch.empty(T, n, dtype=BF, device="cuda") for n in widths[1:]]
    x = torch.zeros(T, widths[0], dtype=BF, device="cuda")
    grads = [torch.zeros(n, k, device="cuda") for k, n in zip(widths, widths[1:])]
    dxs = [torch.empty(T, k, dtype=BF, device="cuda") for k in widths[:-1]]

    def chain(wait):
        at = x
        for layer, y in zip(layers, outs):
            at = layer.forward(at, Y=y)
            wait()
        for layer, d, g in zip(layers[::-1], dxs[::-1], grads[::-1]):
            at = layer.backward(at, dX=d, dW=g)[0]
            wait()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(lambda: None)
    for seed in range(20):
        x.copy_(_randn(100 + seed, T, widths[0]))
        chain(torch.cuda.synchronize)
        want = [t.clone() for t in (*outs, *dxs, *grads)]
        for t in (*outs, *dxs, *grads):
            t.fill_(7)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((*outs, *dxs, *grads), want)), seed
        for t in (*outs, *dxs, *grads):
            t.fill_(7)
        chain(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip((*outs, *dxs, *grads), want)), seed


def _layer(T, K, N, out):
    """Forward and backward of one layer against their products."""
    X, W, dY = _randn(1, T, K), _randn(2, N, K, std=K ** -0.5), _randn(3, T, N, std=1e-2)
    X[:, :: max(1, K // 5)] *= 30  # uneven blocks
    plan = mlpb.Linear8(T, K, N, out_dtype=out)
    plan.load(W)
    w = _values(W, True)
    _check(plan.forward(X), _values(X), w)
    dX, dW = plan.backward(dY)
    _check(dX, _values(dY), w.t())
    _check(dW, _transposed(dY), _transposed(X))
    assert mlpb.mlpb_linear8_last_device_error(plan.handle) == mlpb.MLPB_OK


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("T,K,N", [
    (2057, 4104, 2312),   # results from registers, in all three products or in two
    (4100, 5120, 1096),
    (4999, 2312, 5128),
    (2100, 8328, 2056),   # more k-blocks than an fp32 sum takes at once
    (8300, 1288, 2312)])  # the same in dW
def test_long_sums_from_registers(T, K, N, out):
    _layer(T, K, N, out)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("K,N", [(5120, 344), (3592, 1032), (11008, 264), (7816, 4096),
                                 (20480, 136)])
@pytest.mark.parametrize("T", [1, 16, 77, 128])
def test_ranges_of_a_long_sum(T, K, N, out):
    """Few tokens: K (and, for dX with the sides exchanged, N) in up to eight ranges, of as many or
    of uneven numbers of blocks, longer than a CTA's ring."""
    _layer(T, K, N, out)
    _layer(T, N, K, out)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("T,K,N", [(500, 5120, 5000), (300, 3080, 4104), (1000, 4616, 2312),
                                   (3100, 1000, 1096), (700, 512, 3080), (250, 6152, 2056)])
def test_few_tiles(T, K, N, out):
    _layer(T, K, N, out)


@pytest.mark.parametrize("T,K,N", [(8, 2 ** 20, 8), (5, 8, 2 ** 20), (300, 2 ** 20, 16),
                                   (300, 16, 2 ** 20), (1, 2 ** 20, 264)])
def test_the_longest_sides(T, K, N):
    _layer(T, K, N, F32)
    _layer(T, K, N, BF)
