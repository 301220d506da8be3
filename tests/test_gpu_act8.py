"""GPU parity of the 8-bit activation checkpoints (mlpb_act8_save / mlpb_act8_grad, and
MLPB_FLAG_CHECKPOINT8 of the block) against the fp64 oracle.

Codes and scales are exact (every step of the quantization is).  The activations are bf16
roundings of fp32 evaluations.  Tolerances: half a bf16 step (2^-8 of the value) for the
rounding, and 4e-5 of the magnitude of the terms summed for the evaluation: the sigmoid is
1 / (1 + e^x) with a hardware exponential of relative error <= 2^-22 plus 2^-23 |x| from the
rounded argument, |x| <= 100 for any value that is not yet 0 or 1: 1.2e-5, and a few more
2^-23 for the divide and the products.  A sigmoid below 2^-126 comes out as zero (the fast
divide gives 0 for divisors above 2^126); the factors it meets are at most |dA| < 6 and
|u|, 1 + |g| < 160 here (30 times 1.3 times a normal value below 4.1), 6 * 160 * 160 < 2^18:
values under 2^-126 2^18 = 2^-108 may be lost.
"""
import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from inputs import MLPShape, WORKLOADS, make_inputs, reduced_tokens
from oracle import act8
from oracle.mlp import sigmoid

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8
EVAL = 4e-5
TINY = 2.0 ** -108

# (tokens, ffn, tp): one token, one block and less, short last blocks, several shards,
# columns past one CTA, rows past one CTA's
SHAPES = [(1, 8, 1), (1, 32, 1), (3, 40, 1), (5, 120, 3), (77, 1032, 3), (130, 2048, 8),
          (33, 64, 8), (1000, 96, 2), (6, 20480, 8), (9, 11008, 8)]


def _inputs(T, F, act, seed, special=True):
    g = torch.Generator().manual_seed(seed)
    f1 = 2 * F if act == "swiglu" else F
    z = 1.3 * torch.randn(T, f1, generator=g)
    if special and T >= 3:
        z[0] = 0.0                                   # blocks of zeros
        z[1] *= 30.0                                 # where the sigmoid saturates
        z[2] *= torch.exp2(torch.randint(-12, 3, (f1,), generator=g).float())
    dA = torch.randn(T, F, generator=g)
    return z.to(torch.bfloat16), dA.to(torch.bfloat16)


def _close(name, got, ref, terms):
    """|got - ref| within a rounding of the value and EVAL of the terms it is summed from."""
    got = got.double().cpu().numpy()
    bound = HALF_STEP * np.abs(ref) + 1.01 * EVAL * terms + TINY
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (name, np.abs(got - ref)[bad].max(), int(bad.sum()))


def _terms(dA, z, F, tp, act):
    """Magnitudes of the terms that A and dZ are summed from."""
    if act == "gelu":
        s = sigmoid(2 * 0.7978845608028654 * (z + 0.044715 * z ** 3))
        d = np.abs(2 * 0.7978845608028654 * z * (1 + 3 * 0.044715 * z * z))
        return np.abs(z) * s, np.abs(dA) * (s + d * s * (1 - s) + d * s * 2.0 ** -9)
    g, u = act8._gate_up(z, F, tp)
    d = np.abs(dA).reshape(g.shape)
    s = sigmoid(g)
    a = np.abs(g * u) * s
    dg = d * np.abs(u) * s * (1 + np.abs(g) * (1 - s) + np.abs(g) * 2.0 ** -9)
    return a.reshape(dA.shape), np.stack([dg, d * np.abs(g) * s], 2).reshape(z.shape)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("T,F,tp", SHAPES)
def test_save_and_grad(T, F, tp, act):
    z, dA = _inputs(T, F, act, T + F)
    ck = mlpb.ActCheckpoint8(T, F, tp, act)
    ck.codes.fill_(99)
    ck.scales.fill_(77)
    A = ck.save(z.cuda())
    dZ, A2 = ck.grad(dA.cuda())
    torch.cuda.synchronize()
    zo, do = z.double().numpy(), dA.double().numpy()
    codes, scales = act8.quantize(zo, F, tp, act)
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    assert np.array_equal(ck.scales.cpu().numpy(), scales)
    zh = act8.decode(codes, scales, F, tp, act)
    ta, _ = _terms(do, zo, F, tp, act)
    _close("A", A, act8.act(zo, F, tp, act), ta)
    ta, tz = _terms(do, zh, F, tp, act)
    _close("A again", A2, act8.act(zh, F, tp, act), ta)
    _close("dZ", dZ, act8.act_grad(do, zh, F, tp, act), tz)


def test_without_the_activation_output():
    z, dA = _inputs(5, 120, "swiglu", 3)
    full, part = (mlpb.ActCheckpoint8(5, 120, 3, "swiglu") for _ in range(2))
    full.save(z.cuda())
    mlpb.mlpb_act8_save("swiglu", z.cuda(), None, part.codes, part.scales, 3)
    assert torch.equal(full.codes, part.codes) and torch.equal(full.scales, part.scales)
    want, _ = full.grad(dA.cuda())
    got = torch.empty_like(want)
    mlpb.mlpb_act8_grad("swiglu", dA.cuda(), part.codes, part.scales, got, None, 3)
    assert torch.equal(want, got)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_extreme_values(act):
    """Borders of the scale, the type's extremes, and blocks with infinities and NaN."""
    F = 64
    f1 = 2 * F if act == "swiglu" else F
    z = torch.zeros(8, f1)
    z[0, 3] = 2.0 ** -133
    z[1, :2] = torch.tensor([127.0, 126.5])
    z[2, 0] = 127.5
    z[3] = 3.3e38
    z[4, 5] = float("inf")
    z[5, 40] = float("nan")
    z[6, 33] = -float("inf")
    z[7] = torch.linspace(-3, 3, f1)
    z = z.to(torch.bfloat16)
    ck = mlpb.ActCheckpoint8(8, F, 1, act)
    ck.save(z.cuda())
    dA = torch.ones(8, F, dtype=torch.bfloat16, device="cuda")
    dZ, A = ck.grad(dA)
    codes, scales = act8.quantize(z.double().numpy(), F, 1, act)
    assert np.array_equal(ck.scales.cpu().numpy(), scales)
    finite = np.repeat(scales != 255, 32, axis=1)
    assert np.array_equal(ck.codes.cpu().numpy()[finite], codes[finite])
    # a block with a non-finite value gives NaN gradients in all its places, and no other does
    lost = ~finite
    if act == "swiglu":
        lost = lost.reshape(8, 2, F).any(1, keepdims=True).repeat(2, 1).reshape(8, f1)
    got = torch.isnan(dZ).cpu().numpy()
    got[3] = lost[3]  # 3.3e38 squared is out of fp32's range: no statement
    assert np.array_equal(got, lost)


def test_no_tokens_other_stream_and_graph():
    empty = mlpb.ActCheckpoint8(0, 64, 1, "gelu")
    assert empty.save(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")).shape == (0, 64)
    z, dA = (t.cuda() for t in _inputs(77, 1032, "swiglu", 11))
    ck = mlpb.ActCheckpoint8(77, 1032, 3, "swiglu")
    A = ck.save(z).clone()
    dZ = ck.grad(dA)[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ck2 = mlpb.ActCheckpoint8(77, 1032, 3, "swiglu")
    with torch.cuda.stream(s):
        A2 = ck2.save(z)
    assert torch.equal(A2, A) if s.synchronize() is None else False
    zin, out = torch.zeros_like(z), torch.empty_like(dZ)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ck2.save(zin, A2)
        ck2.grad(dA, out, A2)
    zin.copy_(z)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, dZ) and torch.equal(ck2.codes, ck.codes)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_offsets_past_32_bits(act):
    """The last rows of 2^32 values and more."""
    F = 32768
    f1 = 2 * F if act == "swiglu" else F
    T, n = 2 ** 32 // f1 + 24, 5
    z, dA = _inputs(n, F, act, 7, special=False)
    Z = torch.zeros(T, f1, dtype=torch.bfloat16, device="cuda")
    D = torch.zeros(T, F, dtype=torch.bfloat16, device="cuda")
    Z[-n:], D[-n:] = z.cuda(), dA.cuda()
    big, small = mlpb.ActCheckpoint8(T, F, 1, act), mlpb.ActCheckpoint8(n, F, 1, act)
    A, a = big.save(Z), small.save(z.cuda())
    assert torch.equal(A[-n:], a) and (A[:-n] == 0).all()
    assert torch.equal(big.codes[-n:], small.codes) and torch.equal(big.scales[-n:], small.scales)
    del Z
    dZ, A2 = big.grad(D)
    dz, a2 = small.grad(dA.cuda())
    assert torch.equal(dZ[-n:], dz) and torch.equal(A2[-n:], a2)


def test_refusals():
    z = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    ck = mlpb.ActCheckpoint8(4, 64, 1, "gelu")
    A = torch.empty_like(z)
    for bad in (z[:, :32], z.t().contiguous().t(), z.float()):
        with pytest.raises((ValueError, TypeError, mlpb.MLPBError)):
            mlpb.mlpb_act8_save("gelu", bad, A, ck.codes, ck.scales)
    with pytest.raises(ValueError):
        mlpb.mlpb_act8_save("gelu", z, A, ck.codes, ck.scales[:, :1])
    with pytest.raises(TypeError):
        mlpb.mlpb_act8_save("gelu", z, A, ck.codes.view(torch.uint8), ck.scales)
    with pytest.raises(ValueError):
        mlpb.mlpb_act8_save("swiglu", torch.zeros(4, 65, dtype=torch.bfloat16, device="cuda"),
                            None, ck.codes, ck.scales, 1)


# ------------------------------------------------------------------ the block's flag
BLOCKS = [
    pytest.param(MLPShape(384, 320, 1408, 4, "gelu", True), 81, id="gelu-t4-bias"),
    pytest.param(MLPShape(128, 192, 640, 1, "gelu", False), 83, id="gelu-t1"),
    pytest.param(MLPShape(256, 192, 768, 8, "swiglu", False), 82, id="swiglu-t8-Fs96"),
    pytest.param(reduced_tokens(WORKLOADS[3], 512), 3, id="gelu-H5120-F20480-t8-T512"),
    pytest.param(reduced_tokens(WORKLOADS[4], 512), 4, id="swiglu-H4096-F11008-t8-T512"),
]


def _step(shape, g, flags, z=None, poison=False):
    blk = mlpb.MLPBlock(shape.tokens, shape.hidden, shape.ffn, shape.tp, shape.act, shape.bias,
                        flags=flags)
    out = {"Y": blk.forward(g["X"], g["W1"], g["b1"], g["W2"], g["b2"])}
    out["A"] = blk.A.clone()
    if z is not None:
        blk.Z.copy_(z)
    out["Z"] = blk.Z.clone()
    if poison:
        blk.A.fill_(float("nan"))
    out["grads"] = blk.backward(g["X"], g["W1"], g["W2"], g["dY"])
    torch.cuda.synchronize()
    assert mlpb.mlpb_last_device_error(blk.handle) == 0
    blk.close()
    return out


@pytest.mark.parametrize("shape,wid", BLOCKS)
def test_block_with_checkpoints(shape, wid):
    """The flag changes what is saved and nothing else: the forward is the plain block's bit
    for bit, the codes are those of its Z, and the gradients are, bit for bit, those that the
    recomputing block gives for the values the codes stand for (which bf16 holds exactly)."""
    d = make_inputs(shape, wid)
    g = {k: (v.cuda() if v is not None else None) for k, v in d.items()}
    got = _step(shape, g, mlpb.MLPB_FLAG_CHECKPOINT8, poison=True)
    plain = _step(shape, g, mlpb.MLPB_FLAG_RECOMPUTE_ACT)
    assert torch.equal(got["Y"], plain["Y"]) and torch.equal(got["A"], plain["A"])
    T, F, f1 = shape.tokens, shape.ffn, shape.f1
    codes = got["Z"][:T * f1].view(torch.int8).view(T, f1)
    scales = got["Z"][T * f1:].view(T, f1 // 32)
    ck = mlpb.ActCheckpoint8(T, F, shape.tp, shape.act)
    ck.save(plain["Z"])  # the standalone operator is checked against the oracle above
    assert torch.equal(ck.codes, codes) and torch.equal(ck.scales, scales)
    rows = [0, T // 2, T - 1]
    want = act8.quantize(plain["Z"][rows].double().cpu().numpy(), F, shape.tp, shape.act)
    assert np.array_equal(codes[rows].cpu().numpy(), want[0])
    zh = (codes.float().view(T, -1, 32) * torch.exp2(scales.float() - 127)[..., None]).view(T, f1)
    assert torch.equal(zh.to(torch.bfloat16).float(), zh)
    ref = _step(shape, g, mlpb.MLPB_FLAG_RECOMPUTE_ACT, z=zh.to(torch.bfloat16))
    for k, v in ref["grads"].items():
        assert v is None or torch.equal(v, got["grads"][k]), k
    # and they are close to the uncompressed block's: each value moved by at most half a step
    # of its block, 2^-7 of the block's largest
    for k in ("dW1", "dW2", "dX"):
        a, b = got["grads"][k], plain["grads"][k]
        assert ((a - b).norm() / b.norm()).item() < 2.0 ** -6, k


def test_block_flags_together():
    """With accumulation, bf16 outputs and the emulated exchange, as without them."""
    shape = MLPShape(256, 192, 512, 2, "swiglu", False, True)
    d = make_inputs(shape, 84)
    g = {k: (v.cuda() if v is not None else None) for k, v in d.items()}
    flags = (mlpb.MLPB_FLAG_CHECKPOINT8 | mlpb.MLPB_FLAG_ACCUMULATE_GRADS
             | mlpb.MLPB_FLAG_BF16_OUT | mlpb.MLPB_FLAG_EMULATE_COPIES)
    args = (shape.tokens, shape.hidden, shape.ffn, shape.tp, shape.act, False)
    one = mlpb.MLPBranch(*args, flags=mlpb.MLPB_FLAG_CHECKPOINT8)
    two = mlpb.MLPBranch(*args, flags=flags)
    ya = one.forward(g["X"], g["gamma"], g["beta"], g["W1"], None, g["W2"], None)
    yb = two.forward(g["X"], g["gamma"], g["beta"], g["W1"], None, g["W2"], None)
    ga = one.backward(g["X"], g["gamma"], g["W1"], g["W2"], g["dY"])
    gb = two.backward(g["X"], g["gamma"], g["W1"], g["W2"], g["dY"])
    assert torch.equal(ya.to(torch.bfloat16), yb)
    assert torch.equal(ga["dW1"], gb["dW1"]) and torch.equal(ga["dW2"], gb["dW2"])
    for b in (one, two):
        assert mlpb.mlpb_last_device_error(b.handle) == 0
        b.close()
