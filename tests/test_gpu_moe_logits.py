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
