"""GELU's slope over the whole range of finite inputs: 0 and 1 far out, never NaN, in the 8-bit
checkpoints' gradient and in the block's backward.

For |z| >= 16 the sigmoid of the tanh form is 0 or 1 to far below fp32's last bit, so the slope is
exactly 0 or 1, dZ exactly 0 or dA, and A exactly 0 or z (all bf16 values).
"""
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
# past fp32's range: z^3 from 7e12 on, z^2 from 1.8e19 on
FAR = [16.0, 1e4, 1e12, 6e12, 1.1e13, 1.3e13, 2e13, 1e17, 1.8e19, 2e19, 1e30, 1e38, 3.3e38]


def test_checkpoint_gradient():
    z = torch.tensor([s * v for v in FAR for s in (1, -1)]).to(BF)
    Z = z[:, None].repeat(1, 64).contiguous()
    ck = mlpb.ActCheckpoint8(len(z), 64)
    A = ck.save(Z.cuda()).cpu()
    zh = (ck.codes.cpu().double()
          * torch.exp2(ck.scales.cpu().double() - 127).repeat_interleave(32, 1)).to(BF)
    dA = torch.full((len(z), 64), -1.5, dtype=BF)
    dZ, A2 = (t.cpu() for t in ck.grad(dA.cuda()))
    up = (Z > 0)
    assert torch.equal(dZ, torch.where(up, dA, 0))
    assert torch.equal(A, torch.where(up, Z, 0)) and torch.equal(A2, torch.where(up, zh, 0))


@pytest.mark.parametrize("flag", [0, mlpb.MLPB_FLAG_RECOMPUTE_ACT, mlpb.MLPB_FLAG_CHECKPOINT8])
@pytest.mark.parametrize("sign", [1, -1])
def test_block_backward(flag, sign):
    """db1 = sum over tokens of dZ: of dA = dY W2 where z is far above 0, and 0 far below.  The
    inputs are small integers, so dA and its bf16 rounding (below 2^8) and all sums are exact."""
    T, H, F, t = 128, 64, 128, 2
    g = torch.Generator().manual_seed(3)
    X = torch.zeros(T, H).to(BF).cuda()
    W1 = torch.zeros(t, F // t, H).to(BF).cuda()
    W2 = torch.randint(-2, 3, (t, H, F // t), generator=g).to(BF).cuda()
    b1, b2 = torch.zeros(F).to(BF).cuda(), torch.zeros(H).to(BF).cuda()
    dY = torch.randint(-1, 2, (T, H), generator=g).to(BF).cuda()
    dA = torch.einsum("th,ihj->tij", dY.double(), W2.double()).reshape(T, F)
    assert dA.abs().max() <= 256
    want = dA.sum(0) if sign > 0 else torch.zeros_like(dA.sum(0))
    blk = mlpb.MLPBlock(T, H, F, t, "gelu", True, flags=flag)
    for z in FAR:
        blk.forward(X, W1, b1, W2, b2)
        if flag & mlpb.MLPB_FLAG_CHECKPOINT8:  # codes, then scale bytes: 100 steps of 2^e
            e = int(torch.tensor(z / 100).log2().clamp(max=120).floor())
            blk.Z[:T * F] = sign * 100 & 0xff
            blk.Z[T * F:] = 127 + e
        else:
            blk.Z.fill_(sign * z)
        blk.A.zero_()
        db1 = blk.backward(X, W1, W2, dY)["db1"]
        assert torch.equal(db1.double(), want), z
