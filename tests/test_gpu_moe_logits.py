"""The router's sums where every addition loses as much as it can: a logit is within
D = (8 ceil(H / 4096) + 24) u of sum |x||wr| (u = 2^-24), so a weight (a softmax) within 2 D + 16 u.
"""
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16


@pytest.mark.parametrize("T,E", [(16, 16), (1, 16)])  # four warps a pair, and sixteen
@pytest.mark.parametrize("H", [8192, 65536])
@pytest.mark.parametrize("ones", [8, 32])
def test_additions_of_half_a_step(T, E, H, ones):
    """Expert 0's row: ones in every 8th (or 32nd) place of the first 1024, 2^-24 in all others; a sum
    that holds a one loses each of them (half a step, ties to even).  The other experts have the ones
    alone, exact sums."""
    Wr = torch.zeros(E, H)
    Wr[:, :1024:ones] = 1.0
    Wr[0] += 2.0 ** -24 * (Wr[0] == 0)
    Wr = Wr.to(BF)
    X = torch.ones(T, H, dtype=BF)
    plan = mlpb.MoEDecode(T, H, 8, E, E, "gelu", False)
    _, ids, w = plan.forward(X.cuda(), Wr.cuda(), torch.zeros(E, 8, H, dtype=BF, device="cuda"),
                             torch.zeros(E, H, 8, dtype=BF, device="cuda"))
    assert mlpb.mlpb_moe_last_device_error(plan.handle) == 0
    l = (X.double() @ Wr.double().T)
    want = torch.softmax(l, 1).gather(1, ids.cpu().long())
    D = (8 * -(-H // 4096) + 24) * U * l.max().item()
    assert ((w.cpu().double() - want).abs() <= (2 * D + 16 * U) * want).all()


@pytest.mark.parametrize("T,E,K,H", [(64, 256, 16, 1032), (20, 64, 8, 4096), (1, 128, 16, 4104),
                                     (3, 8, 8, 8192)])
def test_near_ties(T, E, K, H):
    """Experts in pairs whose logits differ by 2^-27, far below what fp32 sums resolve (half a step
    of a sum of one is 2^-25 or more): their order is that of the 64-bit logits, which 64-bit sums
    give to 2^-45, and the kernel to 2^-40 sum |x||wr| < 2^-32; and a token alone has the experts
    that it has among others."""
    g = torch.Generator().manual_seed(T + E + H)
    X = torch.randn(T, H, generator=g)
    Wr = torch.randn(E // 2, H, generator=g) * H ** -0.5
    X[:, 5] = torch.randint(0, 2, (T,), generator=g) * 2.0 - 1
    Wr[:, 5] = 2.0 ** -20 * (1 + torch.randint(0, 127, (E // 2,), generator=g) / 128)
    other = Wr.clone()
    other[:, 5] += 2.0 ** -27
    X, Wr = X.to(BF), torch.cat([Wr, other]).to(BF)
    assert (X.double().abs() @ Wr.double().abs().T).max() < 256
    l = X.double() @ Wr.double().T
    want = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :K]
    plan = mlpb.MoEDecode(T, H, 8, E, K, "gelu", False)
    d = (Wr.cuda(), torch.zeros(E, 8, H, dtype=BF, device="cuda"),
         torch.zeros(E, H, 8, dtype=BF, device="cuda"))
    ids, w = plan.forward(X.cuda(), *d)[1:]
    assert mlpb.mlpb_moe_last_device_error(plan.handle) == 0
    assert torch.equal(ids.cpu().long(), want)
    for t in (0, T // 2, T - 1):
        alone = plan.forward(X[t:t + 1].cuda(), *d)
        assert torch.equal(alone[1][0], ids[t])
