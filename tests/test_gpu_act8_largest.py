"""8-bit checkpoints of bf16's largest value: every finite block stands for finite values, each within
half a step of what was saved, and gradients of finite inputs that have finite values are finite."""
import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from oracle import act8

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
MOST = torch.finfo(BF).max


def _rows(f1):
    """The largest value alone, with both signs, among ties (n + 1/2 steps of 2^121) and others, and
    the values next below it."""
    z = torch.zeros(7, f1, dtype=torch.float64)
    z[0, 5] = MOST
    z[1, ::3], z[1, 1::3] = MOST, -MOST
    z[2, :63] = (torch.arange(63) + 0.5) * 2.0 ** 121
    z[2, 63] = -MOST
    z[3, :64] = torch.arange(64) * 2.0 ** 121
    z[3, 40] = MOST
    z[4] = 254 * 2.0 ** 120
    z[5, :32] = -254 * 2.0 ** 120
    z[6] = 2.0 ** 127
    out = z.to(BF)
    assert torch.equal(out.double(), z)
    return out


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_codes(act):
    F = 64
    z = _rows(2 * F if act == "swiglu" else F)
    ck = mlpb.ActCheckpoint8(len(z), F, 1, act)
    ck.save(z.cuda())
    codes, scales = act8.quantize(z.double().numpy(), F, 1, act)
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    assert np.array_equal(ck.scales.cpu().numpy(), scales)
    got = act8.decode(codes, scales, F, 1, act)
    step = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    assert (np.abs(got) <= MOST).all() and (np.abs(got - z.double().numpy()) <= step / 2).all()


def test_gelu_gradient():
    z = _rows(64)
    ck = mlpb.ActCheckpoint8(len(z), 64)
    ck.save(z.cuda())
    zh = torch.from_numpy(act8.decode(*act8.quantize(z.double().numpy(), 64, 1, "gelu"), 64, 1,
                                      "gelu")).to(BF)
    dA = torch.full((len(z), 64), 3.0, dtype=BF)
    dZ, A = (t.cpu() for t in ck.grad(dA.cuda()))
    slope = torch.where(zh > 0, 1.0, torch.where(zh < 0, 0.0, 0.5))
    assert torch.equal(dZ, (dA * slope).to(BF)) and torch.equal(A, zh.clamp(min=0))


def test_swiglu_gradient():
    """A far gate below zero gives zeros; a largest up times a gate of one is finite."""
    z = torch.zeros(2, 128, dtype=BF)
    z[0, :64], z[0, 64:] = -MOST, 1.0
    z[1, :64], z[1, 64:] = 0.5, MOST
    ck = mlpb.ActCheckpoint8(2, 64, 1, "swiglu")
    ck.save(z.cuda())
    dA = torch.ones(2, 64, dtype=BF)
    dZ, A = (t.cpu() for t in ck.grad(dA.cuda()))
    assert (A[0] == 0).all() and (dZ[0] == 0).all()
    assert torch.isfinite(A).all() and torch.isfinite(dZ).all() and (A[1] > 1e37).all()


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_block(act):
    """The block's epilogue writes the same codes: Z = X W1^T with one factor in each sum."""
    T, H, F = 128, 128, 128
    f1 = 2 * F if act == "swiglu" else F
    z = torch.cat([_rows(f1), torch.zeros(T - 7, f1, dtype=BF)])
    X = torch.zeros(T, H, dtype=BF)
    X[:7, :7] = torch.eye(7)
    W1 = torch.zeros(f1, H, dtype=BF)
    W1[:, :7] = z[:7].T
    W1 = W1.view(1, 2, F, H) if act == "swiglu" else W1.view(1, F, H)
    blk = mlpb.MLPBlock(T, H, F, 1, act, False, flags=mlpb.MLPB_FLAG_CHECKPOINT8)
    blk.forward(X.cuda(), W1.cuda(), None, torch.zeros(1, H, F, dtype=BF, device="cuda"), None)
    ck = mlpb.ActCheckpoint8(T, F, 1, act)
    ck.save(z.cuda())
    assert torch.equal(blk.Z[:T * f1].view(torch.int8), ck.codes.view(-1))
    assert torch.equal(blk.Z[T * f1:], ck.scales.view(-1))
