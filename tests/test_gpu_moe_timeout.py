"""Bounded waits of the mixture-of-experts kernel: a launch that misses a stage's weights (an arrival
that nothing makes) or a CTA at a barrier of the grid ends by itself, the handle reports it, and the
next launch is right."""
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# a few tokens an expert (a ring for each group), and more than 16 (one ring for the CTA)
@pytest.mark.parametrize("T,H,F,E,K,act", [(3, 1024, 520, 4, 2, "swiglu"),
                                           (40, 1024, 264, 2, 1, "gelu"),
                                           (64, 2048, 1032, 3, 2, "swiglu")])
def test_expired_waits_are_reported_and_the_next_launch_is_right(T, H, F, E, K, act):
    g = torch.Generator(device="cuda").manual_seed(T + H + F)

    def n(*shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)
    w1 = (E, 2, F, H) if act == "swiglu" else (E, F, H)
    d = (n(T, H, std=1.0), n(E, H, std=H ** -0.5), n(*w1, std=H ** -0.5), n(E, H, F, std=F ** -0.5))
    want = mlpb.MoEDecode(T, H, F, E, K, act).forward(*d)
    torch.cuda.synchronize()
    plan = mlpb.MoEDecode(T, H, F, E, K, act)
    good = plan.handle
    plan.handle = mlpb.mlpb_moe_create(mlpb.make_moe_config(T, H, F, E, K, act,
                                                            flags=mlpb.MLPB_MOE_FAULT_INJECT))
    mlpb.mlpb_moe_destroy(good)
    for _ in range(2):  # a stage that is never filled; a barrier that a CTA misses
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        plan.forward(*d)
        end.record()
        assert mlpb.mlpb_moe_last_device_error(plan.handle) == mlpb.MLPB_ETIMEOUT
        # the waits' limit is 1 s; at most three follow each other (a stage's or the first barrier's,
        # then two barriers'), and no time goes on copies that never come
        assert 900 < start.elapsed_time(end) < 3500
    for _ in range(3):
        out = plan.forward(*d)
        assert mlpb.mlpb_moe_last_device_error(plan.handle) == mlpb.MLPB_OK
        assert all(torch.equal(a, b) for a, b in zip(out, want))
