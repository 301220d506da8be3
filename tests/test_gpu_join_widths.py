"""The join at widths on both sides of its layouts' borders, and the same bits in every call.

Tolerances: those of test_gpu_join.py, whose checks these are.
"""
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from test_gpu_join import BF, F32, _make, _run

pytestmark = pytest.mark.gpu


# four, five and eight warps a row in the forward, by width and norm; the backward's plain and
# general instantiations
@pytest.mark.parametrize("H", [4096, 4104, 4608, 5112, 5120, 5128, 6144, 7168])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), ("rms", "layer"),
                                      ("none", "rms")])
def test_borders(H, post, pre):
    _run(37, H, post, pre, 1, True, BF, BF)
    _run(330, H, post, pre, 330, False, F32, BF)


@pytest.mark.parametrize("T,H,post,pre,G,xt,yt", [
    (600, 8192, "rms", "rms", 1, BF, BF), (900, 4096, "layer", "layer", 9, F32, F32),
    (500, 5112, "layer", "layer", 1, BF, BF), (300, 9856, "rms", "rms", 3, BF, F32),
    (300, 16384, "layer", "rms", 1, BF, BF), (2000, 520, "rms", "rms", 2000, BF, BF)])
def test_every_call_has_the_first_ones_bits(T, H, post, pre, G, xt, yt):
    """Rows are copied ahead into memory that is read at the same time: a copy that came too early
    would give other values now and then."""
    d = _make(T, H, post, pre, G, True, xt, yt)
    plan = mlpb.Join(T, H, post, pre, G, 1e-5, xt, yt)
    par = {k: d[k] for k in ("res_scale", "gate", "gamma_post", "beta_post", "gamma_pre",
                             "beta_pre")}
    first = plan.forward(d["X"], d["Y"], **par)
    grads = plan.backward(d["X"], d["Y"], first[0], first[2], d["dXout"], d["dXn"], **par)
    names = [k for k, v in grads.items() if v is not None]
    out, again = [torch.empty_like(t) for t in first], plan.alloc_grads(True)
    busy = torch.zeros(16 << 20, device="cuda")
    wrong = torch.zeros(3 + len(names), dtype=torch.int64, device="cuda")
    for i in range(200):
        if i % 3 == 0:
            busy.add_(1)
        plan.forward(d["X"], d["Y"], **par, Xout=out[0], Xn=out[1], stats=out[2])
        plan.backward(d["X"], d["Y"], first[0], first[2], d["dXout"], d["dXn"], **par, grads=again)
        wrong += torch.stack([(a != b).sum() for a, b in zip(out, first)]
                             + [(again[k] != grads[k]).sum() for k in names])
    assert not wrong.any(), dict(zip(["Xout", "Xn", "stats"] + names, wrong.tolist()))
