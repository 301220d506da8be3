"""Block-scaled E4M3 and the linear layer on it against the fp64 oracle (oracle/b128.py).

Tolerances.  Codes and scales: none, every value is the oracle's.  Products: a product of two codes
with their scales is exact in fp32; an MMA adds 32 of them to the accumulator, and what its
alignment and the sum cut off is taken as at most 2^-22 of the magnitudes added so far, so that K
products are off by at most (ceil(K / 32) + 4) 2^-22 of the sum of their magnitudes.  A bf16 output
adds half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from oracle import b128

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _randn(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _check(got, want, mags, terms, bf16, base=None):
    tol = (-(-terms // 32) + 4) * 2.0 ** -22 * mags
    if base is not None:
        want = want + base
        tol = tol + 2.0 ** -23 * np.abs(want)  # the addition into what was there
    if bf16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    d = np.abs(_np(got) - want)
    assert (d <= tol + 1e-300).all(), f"{(d - tol).max():.3e} over, {np.count_nonzero(d > tol)}"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("R,C", [(1, 8), (3, 136), (77, 1032), (128, 128), (129, 512), (260, 648)])
def test_quantize(R, C, square, dtype):
    x = _randn(R * C, R, C, dtype=F32)
    x *= torch.exp(4 * _randn(7, R, 1, dtype=F32))
    x[:, :: max(1, C // 5)] *= 1000
    x[R // 2, : min(C, 128)] = 0
    x = x.to(dtype)
    q, qt = mlpb.b128_empty(R, C, "cuda"), mlpb.b128_empty(C, R, "cuda")
    for t in (*q, *qt):
        t.fill_(0xa5)
    mlpb.mlpb_b128_quantize(x, q, qt, square)
    for pair, rows, cols, src in ((q, R, C, _np(x)), (qt, C, R, _np(x).T)):
        want, e = b128.quantize(src, square)
        assert np.array_equal(_np(mlpb.b128_values(pair, rows, cols)), want)
        assert bool((pair[0][:, cols:] == 0).all())
        # the scale bytes where the header says, 127 past the end
        s = pair[1].cpu().numpy()
        tiles, groups = -(-rows // 128), -(-cols // 512)
        for r in (0, rows - 1, tiles * 128 - 1):
            for kb in range(groups * 4):
                at = ((kb // 4) * tiles + r // 128) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + kb % 4
                past = r >= rows or kb * 128 >= cols
                assert s[at] == (127 if past else e[r // (128 if square else 1), kb])
    one = mlpb.b128_empty(R, C, "cuda"), mlpb.b128_empty(C, R, "cuda")
    mlpb.mlpb_b128_quantize(x, one[0], None, square)  # each by itself
    mlpb.mlpb_b128_quantize(x, None, one[1], square)
    assert all(torch.equal(a, b) for a, b in zip((*one[0], *one[1]), (*q, *qt)))


def test_quantize_extremes():
    big = torch.finfo(F32).max
    x = torch.zeros(4, 264, device="cuda")
    x[0, 0], x[0, 5] = big, -big / 3
    x[1, 0], x[1, 1] = 2.0 ** -149, 2.0 ** -130
    x[2, 3] = float("inf")
    x[2, 130] = float("nan")
    x[3, 0], x[3, 1], x[3, 2] = 448.0, 448.0 - 2.0 ** -10, 2.0 ** -9 * 1.5
    q, qt = mlpb.b128_empty(4, 264, "cuda"), mlpb.b128_empty(264, 4, "cuda")
    mlpb.mlpb_b128_quantize(x, q, qt)
    for pair, shape, src in ((q, (4, 264), _np(x)), (qt, (264, 4), _np(x).T)):
        assert np.array_equal(_np(mlpb.b128_values(pair, *shape)), b128.quantize(src)[0],
                              equal_nan=True)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("T,K,N", [(1, 8, 8), (1, 1032, 344), (5, 640, 264), (16, 2056, 136),
                                   (33, 512, 520), (64, 1408, 640), (77, 1032, 344),
                                   (130, 264, 1000), (257, 520, 264), (300, 136, 2056)])
def test_layer(T, K, N, out):
    X = _randn(T + K, T, K) * torch.exp(_randn(1, T, 1))
    X[:, :: max(1, K // 3)] *= 30
    W, dY = _randn(N, N, K, std=K ** -0.5), _randn(N + T, T, N, std=1e-3)
    plan = mlpb.Linear8(T + 3, K, N, out_dtype=out)
    plan.load(W)
    Y = plan.forward(X)
    dX, dW = plan.backward(dY)
    o = b128.linear(_np(X), _np(W), _np(dY))
    _check(Y, *o["Y"], K, out == BF)
    _check(dX, *o["dX"], N, out == BF)
    _check(dW, *o["dW"], T, False)
    was = _randn(3, N, K, dtype=F32, std=0.1)
    acc = was.clone()
    assert plan.backward(dY, dW=acc, accumulate=True, input_grad=False)[0] is None
    _check(acc, *o["dW"], T, False, base=_np(was))
    assert mlpb.mlpb_linear8_last_device_error(plan.handle) == mlpb.MLPB_OK
    serving = mlpb.Linear8(T, K, N, training=False, out_dtype=out)
    serving.load(W.float())  # the same values in fp32
    assert torch.equal(serving.forward(X), Y)
    assert serving.forward(X[:0]).shape == (0, N)


def _scaled(values):
    """What the library stands for as float64: blocks quantized by the oracle's rule, vectorised."""
    x = values.double()
    R, C = x.shape
    b = torch.nn.functional.pad(x, (0, -C % 128)).view(R, -1, 128)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    k = torch.where(m <= 0.875, 9 - e, 8 - e).double()
    q = (b * torch.exp2(k)).float().to(torch.float8_e4m3fn).double() * torch.exp2(-k)
    return q.view(R, -1)[:, :C]


@pytest.mark.parametrize("T,K,N", [(16500, 136, 264), (24700, 264, 8), (9000, 1032, 2056)])
def test_long_sums(T, K, N):
    """dW over more tokens than one sum in the tensor cores: chunks of 64 blocks.  Each chunk's
    error is that of its own length; their additions round, 2^-24 of a partial sum each."""
    X, dY = _randn(1, T, K), _randn(2, T, N, std=1e-3)
    plan = mlpb.Linear8(T, K, N)
    plan.load(_randn(3, N, K))
    plan.forward(X)
    dW = plan.backward(dY, input_grad=False)[1].double()
    a, b = _scaled(dY.t()), _scaled(X.t())
    want, mags = a @ b.t(), a.abs() @ b.abs().t()
    chunks = -(-T // 8192)
    tol = (min(T, 8192) / 32 + 4) * 2.0 ** -22 * mags + chunks * 2.0 ** -24 * mags
    assert bool(((dW - want).abs() <= tol).all())
    # the size of the whole error does not grow with the number of chunks
    assert float((dW - want).norm() / want.norm()) < 1e-6


def test_values_that_are_not_finite_stay_in_their_rows():
    T, K, N = 40, 384, 256
    X, W, dY = _randn(1, T, K), _randn(2, N, K), _randn(3, T, N)
    X[7, 200] = float("inf")
    dY[9, 3] = float("nan")
    plan = mlpb.Linear8(T, K, N)
    plan.load(W)
    Y = plan.forward(X)
    dX, dW = plan.backward(dY)
    o = b128.linear(_np(X), _np(W), _np(dY))
    for got, k in ((Y, "Y"), (dX, "dX"), (dW, "dW")):
        assert np.array_equal(np.isnan(_np(got)), np.isnan(o[k][0])), k
    assert np.isnan(o["Y"][0]).any(1).sum() == 1


def test_large_scales_do_not_meet_in_between():
    """Blocks whose scales are near the ends of the range, whose products are ordinary."""
    T, K, N = 3, 256, 16
    X, W = _randn(1, T, K).float(), _randn(2, N, K).float()
    X[:, :128] *= 2.0 ** 100
    W[:, :128] *= 2.0 ** -100
    X[:, 128:] *= 2.0 ** -90
    W[:, 128:] *= 2.0 ** 90
    plan = mlpb.Linear8(T, K, N, out_dtype=F32)
    plan.load(W)
    o = b128.linear(_np(X.to(BF)), _np(W))
    _check(plan.forward(X.to(BF)), *o["Y"], K, False)


@pytest.mark.parametrize("T", [8, 500, 2056, 4104, 8200, 16500])
def test_gradients_are_added_into_what_is_there(T):
    # tiles for all SMs: both ways take the same products in the same order
    n = 2056
    X, dY, W = _randn(1, T, n), _randn(2, T, n), _randn(3, n, n)
    plan = mlpb.Linear8(T, n, n)
    plan.load(W)
    plan.forward(X)
    dW = plan.backward(dY, input_grad=False)[1].double()
    base = _randn(4, n, n, std=T ** 0.5).float()
    acc = base.clone()
    plan.backward(dY, dW=acc, accumulate=True, input_grad=False)
    # one rounding for each chunk of 8192 tokens and side, of no more than twice the sum of sizes
    # (|dW| is some T^0.5, and so is a chunk's)
    chunks = -(-T // 8192)
    size = base.double().abs() + dW.abs() + (0.0 if chunks == 1 else 6 * T ** 0.5)
    assert bool(((acc.double() - (base.double() + dW)).abs() <= (2 * chunks - 1) * 2.0 ** -24
                 * size * 1.0001).all())


def test_zero_tokens_and_refusals():
    K, N = 64, 48
    plan = mlpb.Linear8(4, K, N)
    plan.load(_randn(1, N, K))
    dW = torch.ones(N, K, device="cuda")
    plan.backward(_randn(2, 0, N), dW=dW, accumulate=True)
    assert bool((dW == 1).all())
    plan.backward(_randn(2, 0, N), dW=dW)
    assert bool((dW == 0).all())
    X, dY = _randn(3, 4, K), _randn(4, 4, N)
    with pytest.raises(mlpb.MLPBError):
        plan.forward(_randn(3, 5, K))  # more than max_tokens
    with pytest.raises(ValueError, match="shape"):
        plan.forward(_randn(3, 4, K + 8))
    with pytest.raises(ValueError, match="contiguous"):
        plan.forward(_randn(3, K, 4).t())
    with pytest.raises(TypeError):
        plan.forward(X.float())
    with pytest.raises(ValueError, match="shape"):
        plan.load(_randn(1, K, N))
    with pytest.raises(ValueError, match="nothing given"):
        plan.backward(dY, accumulate=True)
    with pytest.raises(ValueError, match="training"):
        mlpb.Linear8(4, K, N, training=False).backward(dY)
    with pytest.raises(ValueError, match="last forward"):  # none yet
        plan.backward(dY)
    plan.forward(X[:3])
    with pytest.raises(ValueError, match="4 tokens, the last forward had 3"):
        plan.backward(dY)
    h, Y = plan.handle, torch.empty(4, N, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="are needed"):
        mlpb.mlpb_linear8_forward(h, X, plan.Wq, Y, None, plan.workspace[:16])
    with pytest.raises(mlpb.MLPBError):
        mlpb.mlpb_linear8_forward(h, X, plan.Wq, Y, None, None)
    with pytest.raises(mlpb.MLPBError):
        mlpb.mlpb_linear8_forward(h, X, None, Y, None, plan.workspace)
    with pytest.raises(mlpb.MLPBError):  # neither gradient
        mlpb.mlpb_linear8_backward(h, dY, plan.Wt, plan.saved(4), None, None, False, plan.workspace)
    with pytest.raises(mlpb.MLPBError):  # a misaligned output
        mlpb.mlpb_linear8_forward(h, X, plan.Wq, torch.empty(4 * N + 4, dtype=BF, device="cuda")
                                  [4:].view(4, N), None, plan.workspace)


def test_rows_behind_the_last_are_left_as_they_were():
    T, K, N = 21, 264, 392
    plan = mlpb.Linear8(64, K, N)
    plan.load(_randn(1, N, K))
    for dtype_rows in (T, 64):
        Y = torch.full((64, N), 7.0, dtype=BF, device="cuda")
        plan.forward(_randn(2, dtype_rows, K), Y=Y[:dtype_rows])
        assert bool((Y[dtype_rows:] == 7).all())


def test_graph_another_stream_and_two_plans():
    T, K, N = 70, 520, 264
    X, W, dY = _randn(1, T, K), _randn(2, N, K), _randn(3, T, N)
    plan = mlpb.Linear8(T, K, N)
    plan.load(W)
    want = (plan.forward(X), *plan.backward(dY))
    bufs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    x, d = torch.zeros_like(X), torch.zeros_like(dY)
    with torch.cuda.graph(graph):
        plan.load(W)
        plan.forward(x, Y=bufs[0])
        plan.backward(d, dX=bufs[1], dW=bufs[2])
    x.copy_(X)
    d.copy_(dY)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(bufs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mlpb.Linear8(T, K, N)
    torch.cuda.synchronize()
    other.load(W, stream=side)
    y = other.forward(X, stream=side)
    g = other.backward(dY, stream=side)
    again = (plan.forward(X), *plan.backward(dY))  # beside it on the current stream
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, *g), want))
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_a_saved_transpose_of_ones_own():
    """Two forwards whose backwards come later, each with the X^T that it was given."""
    T, K, N = 24, 136, 72
    plan = mlpb.Linear8(T, K, N)
    plan.load(_randn(1, N, K))
    a, b, dY = _randn(2, T, K), _randn(3, 9, K), _randn(4, T, N)
    kept = mlpb.b128_empty(K, T, "cuda")
    plan.forward(a)
    want = plan.backward(dY)
    plan.forward(a, Xt=kept)
    plan.forward(b)
    got = plan.backward(dY, Xt=kept)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_an_expired_wait_is_reported_and_the_next_call_is_right():
    T, K, N = 300, 640, 520
    X, W = _randn(1, T, K), _randn(2, N, K)
    plan = mlpb.Linear8(T, K, N, training=False)
    plan.load(W)
    want = plan.forward(X)
    hurt = mlpb.Linear8(T, K, N, training=False, flags=mlpb.MLPB_LINEAR8_FAULT_INJECT)
    hurt.load(W)
    hurt.forward(X)
    assert mlpb.mlpb_linear8_last_device_error(hurt.handle) == mlpb.MLPB_ETIMEOUT
    assert torch.equal(hurt.forward(X), want)
    assert mlpb.mlpb_linear8_last_device_error(hurt.handle) == mlpb.MLPB_OK


def test_the_rows_of_an_earlier_forward_are_named():
    """Forward into the plan, forward into an Xt, and both backwards after them."""
    T, K, N = 40, 136, 72
    plan = mlpb.Linear8(T, K, N)
    plan.load(_randn(1, N, K))
    a, b, da, db = _randn(2, T, K), _randn(3, T, K), _randn(4, T, N), _randn(5, T, N)
    plan.forward(a)
    want_a = plan.backward(da)
    plan.forward(b)
    want_b = plan.backward(db)
    plan.forward(a)
    kept = mlpb.b128_empty(K, T, "cuda")
    plan.forward(b, Xt=kept)
    with pytest.raises(ValueError, match="kept no rows here"):
        plan.backward(db)
    got_b = plan.backward(db, Xt=kept)
    got_a = plan.backward(da, Xt=plan.saved(T))
    assert all(torch.equal(p, q) for p, q in zip((*got_a, *got_b), (*want_a, *want_b)))


def test_one_gradient_alone():
    T, K, N = 50, 264, 136
    plan = mlpb.Linear8(T, K, N)
    plan.load(_randn(1, N, K))
    X, dY = _randn(2, T, K), _randn(3, T, N)
    plan.forward(X)
    dX, dW = plan.backward(dY)
    a, none = plan.backward(dY, weight_grad=False)
    assert none is None and torch.equal(a, dX)
    none, b = plan.backward(dY, input_grad=False)
    assert none is None and torch.equal(b, dW)
    # dX needs no rows of a forward: none of this plan, and of another number of tokens
    fresh = mlpb.Linear8(T, K, N)
    fresh.load(_randn(1, N, K))
    assert torch.equal(fresh.backward(dY[:17], weight_grad=False)[0], dX[:17])
    with pytest.raises(ValueError, match="neither gradient"):
        plan.backward(dY, input_grad=False, weight_grad=False)
    a, b = torch.zeros_like(dX), torch.zeros_like(dW)  # given ones are computed all the same
    got = plan.backward(dY, dX=a, dW=b, input_grad=False, weight_grad=False)
    assert got[0] is a and got[1] is b and torch.equal(a, dX) and torch.equal(b, dW)
    with pytest.raises(ValueError, match="nothing given"):
        plan.backward(dY, accumulate=True, weight_grad=False)
