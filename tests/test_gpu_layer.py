"""The operators around and in place of the block, one after the other as a layer uses them: a
training step of two MLP sub-blocks (join, block with 8-bit checkpoints, join, ...) forward and
backward, and a serving step of two mixture-of-experts sub-blocks (join, experts, join, ...).

Every stage is checked against its fp64 oracle on the inputs that the stage before it stored,
with that operator's own tolerances.  The whole chain's gradients are checked against
differences of the plain fp64 chain.  Between the two lie, for each sub-block: the bf16
roundings of Xn, A, dY and dZ (2^-8 of a value each, 2^-8 of the tensor's norm at most), the
code of Z (half a step of 2^-7 of its block's largest, which is below 4 times the block's root
mean square for 32 normal values: 2^-6), and those of Y, Xn and A once more where the backward
reads them: 7 2^-8 + 2^-6 < 2^-4.5 of the branch's gradient, which is half of dX at most here;
dX passes two sub-blocks and a branch parameter's gradient at most two: 2^-3.5.
"""
import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
import test_gpu_join as tj
import test_gpu_moe as tm
from _harness import compare
from oracle import act8, join

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
T, H, F, TP, EPS = 256, 192, 512, 1, 1e-5


def _params(act, seed):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std=1.0, mean=0.0, dtype=BF):
        return (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()
    f1 = 2 * F if act == "swiglu" else F
    return dict(
        X=n(T, H, dtype=F32), dOut=n(T, H, dtype=F32),
        g0=n(H, std=0.1, mean=1.0), g1=n(H, std=0.1, mean=1.0), p1=n(H, std=0.1, mean=1.0),
        p2=n(H, std=0.1, mean=1.0), c2=n(H, std=0.1), gate=n(2, H, std=0.2, mean=0.5),
        W1=[n(f1, H, std=H ** -0.5).view((1, 2, F, H) if act == "swiglu" else (1, F, H))
            for _ in range(2)],
        W2=[n(1, H, F, std=F ** -0.5) for _ in range(2)])


class _Layers:
    """Two sub-blocks; owns nothing that step() computes but what the plans hold."""

    def __init__(self, act):
        args = (T, H, F, TP, act, False)
        self.b = [mlpb.MLPBlock(*args, flags=mlpb.MLPB_FLAG_CHECKPOINT8) for _ in range(2)]
        kw = dict(eps=EPS, stream_dtype=F32, block_dtype=F32)
        self.j0 = mlpb.Join(T, H, "none", "rms", has_block=False, **kw)
        self.j1 = mlpb.Join(T, H, "rms", "rms", gate_groups=2, **kw)
        self.j2 = mlpb.Join(T, H, "layer", "none", **kw)

    def step(self, p):
        r = {}
        _, r["Xn0"], r["s0"] = self.j0.forward(p["X"], gamma_pre=p["g0"])
        r["Y0"] = self.b[0].forward(r["Xn0"], p["W1"][0], None, p["W2"][0], None)
        k1 = dict(gate=p["gate"], gamma_post=p["p1"], gamma_pre=p["g1"])
        r["X1"], r["Xn1"], r["s1"] = self.j1.forward(p["X"], r["Y0"], **k1)
        r["Y1"] = self.b[1].forward(r["Xn1"], p["W1"][1], None, p["W2"][1], None)
        k2 = dict(gamma_post=p["p2"], beta_post=p["c2"])
        r["X2"], _, r["s2"] = self.j2.forward(r["X1"], r["Y1"], **k2)
        r["d2"] = self.j2.backward(r["X1"], r["Y1"], r["X2"], r["s2"], p["dOut"], **k2)
        r["e1"] = self.b[1].backward(r["Xn1"], p["W1"][1], p["W2"][1], r["d2"]["dY"])
        r["d1"] = self.j1.backward(p["X"], r["Y0"], r["X1"], r["s1"], r["d2"]["dX"],
                                   r["e1"]["dX"], **k1)
        r["e0"] = self.b[0].backward(r["Xn0"], p["W1"][0], p["W2"][0], r["d1"]["dY"])
        r["d0"] = self.j0.backward(None, None, p["X"], r["s0"], r["d1"]["dX"], r["e0"]["dX"],
                                   gamma_pre=p["g0"])
        return r

    def close(self):
        for b in self.b:
            assert mlpb.mlpb_last_device_error(b.handle) == 0
            b.close()


def _f64(x):
    return [_f64(v) for v in x] if isinstance(x, list) else x.double().cpu().numpy()


def _act(z, act):
    return act8.act(z, F, TP, act)


def _fc1(x, w):
    return x @ w.reshape(-1, H).T        # one shard: SwiGLU's gates, then its ups


def _loss(p, act):
    """The plain chain in 64 bits."""
    n = join.norm
    x = p["X"]
    y = _act(_fc1(n(x, "rms", EPS)[0] * p["g0"], p["W1"][0]), act) @ p["W2"][0][0].T
    x = x + join.gate_rows(p["gate"], T) * n(y, "rms", EPS)[0] * p["p1"]
    y = _act(_fc1(n(x, "rms", EPS)[0] * p["g1"], p["W1"][1]), act) @ p["W2"][1][0].T
    x = x + n(y, "layer", EPS)[0] * p["p2"] + p["c2"]
    return (x * p["dOut"]).sum()


def _block_check(p, i, act, xn, y, dy, got, codes):
    """One block's outputs for the inputs that were stored, its backward for the codes."""
    x, w1, w2 = _f64(xn), _f64(p["W1"][i]), _f64(p["W2"][i])[0]
    z = _fc1(x, w1)
    compare("Y", _f64(y), _act(z, act) @ w2.T)
    f1 = z.shape[1]
    q = codes[:T * f1].view(torch.int8).view(T, -1, 32).double().cpu().numpy()
    s = codes[T * f1:].view(T, -1).double().cpu().numpy()
    zh = (q * 2.0 ** (s - 127)[..., None]).reshape(T, f1)
    dYf = _f64(dy)
    dZ = act8.act_grad(dYf @ w2, zh, F, TP, act)
    compare("dW2", _f64(got["dW2"])[0], dYf.T @ _act(zh, act))
    compare("dW1", _f64(got["dW1"]).reshape(-1, H), dZ.T @ x)
    compare("dX", _f64(got["dX"]), dZ @ w1.reshape(-1, H))


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_training_step(act):
    p = _params(act, 11)
    m = _Layers(act)
    r = m.step(p)
    torch.cuda.synchronize()
    none = dict(res_scale=None, gate=None, gamma_post=None, beta_post=None, gamma_pre=None,
                beta_pre=None, Y=None)
    d1 = {**none, "X": p["X"], "Y": r["Y0"], "gate": p["gate"], "gamma_post": p["p1"],
          "gamma_pre": p["g1"], "dXout": r["d2"]["dX"], "dXn": r["e1"]["dX"]}
    tj._forward_checks(d1, "rms", "rms", F32, (r["X1"], r["Xn1"], r["s1"]))
    tj._backward_checks(d1, "rms", "rms", F32, r["X1"], r["d1"])
    d2 = {**none, "X": r["X1"], "Y": r["Y1"], "gamma_post": p["p2"], "beta_post": p["c2"],
          "dXout": p["dOut"], "dXn": None}
    tj._forward_checks(d2, "layer", "none", F32, (r["X2"], None, r["s2"]))
    tj._backward_checks(d2, "layer", "none", F32, r["X2"], r["d2"])
    for i, dY in ((0, r["d1"]["dY"]), (1, r["d2"]["dY"])):
        _block_check(p, i, act, r[f"Xn{i}"], r[f"Y{i}"], dY, r[f"e{i}"], m.b[i].Z)
    # the chain's gradients, each along itself
    f = {k: _f64(v) for k, v in p.items()}
    leaves = [("X", None, r["d0"]["dX"]), ("g0", None, r["d0"]["dgamma_pre"]),
              ("gate", None, r["d1"]["dgate"]), ("p1", None, r["d1"]["dgamma_post"]),
              ("g1", None, r["d1"]["dgamma_pre"]), ("c2", None, r["d2"]["dbeta_post"])]
    leaves += [(k, i, r[f"e{i}"]["d" + k]) for k in ("W1", "W2") for i in range(2)]
    for k, i, grad in leaves:
        grad = _f64(grad)
        size = np.linalg.norm(grad)
        v, t = grad / size, 1e-4

        def at(h):
            q = dict(f)
            if i is None:
                q[k] = f[k] + h * v.reshape(f[k].shape)
            else:
                q[k] = list(f[k])
                q[k][i] = f[k][i] + h * v.reshape(f[k][i].shape)
            return _loss(q, act)
        slope = (at(t) - at(-t)) / (2 * t)
        assert abs(slope - size) <= 2.0 ** -3.5 * size, (k, i, slope, size)
    m.close()


def _tensors(r):
    return [t for v in r.values() for t in (v.values() if isinstance(v, dict) else [v])
            if t is not None]


def test_training_step_captured():
    """The step replayed from a graph, on new inputs, gives an eager step's bits."""
    p, q = _params("swiglu", 11), _params("swiglu", 12)
    m, e = _Layers("swiglu"), _Layers("swiglu")
    want = [[t.clone() for t in _tensors(e.step(x))] for x in (p, q)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step(p)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = m.step(p)
    for src, ref in ((p, want[0]), (q, want[1])):
        for k, v in src.items():
            for a, b in zip(*((x if isinstance(x, list) else [x]) for x in (p[k], v))):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(_tensors(r), ref):
            assert torch.equal(a, b)
    del graph
    for x in (m, e):
        x.close()


MT, MH, MF, ME, MK = 16, 264, 72, 12, 3


class _Serve:
    def __init__(self):
        self.moe = [mlpb.MoEDecode(MT, MH, MF, ME, MK) for _ in range(2)]

    def step(self, X, d):
        """X is updated in place; returns what every stage stored."""
        n, keep = X.shape[0], []
        _, xn, _ = mlpb.Join(n, MH, "none", "rms", has_block=False).forward(X, gamma_pre=d["g"][0])
        for i in range(2):
            x_in = X.clone()
            out = self.moe[i].forward(xn, *d["w"][i])
            last = i == 1
            plan = mlpb.Join(n, MH, "rms", "none" if last else "layer")
            par = dict(gamma_post=d["p"][i], gamma_pre=None if last else d["g"][1],
                       beta_pre=None if last else d["b"])
            got = plan.forward(X, out[0], Xout=X, **par)
            keep.append((x_in, xn, out, par, (X.clone(), *got[1:])))
            xn = got[1]
        return keep


def _serve_params():
    g = torch.Generator().manual_seed(5)

    def n(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g) * std + mean).to(BF).cuda()
    w = [(n(ME, MH, std=MH ** -0.5), n(ME, 2, MF, MH, std=MH ** -0.5),
          n(ME, MH, MF, std=MF ** -0.5)) for _ in range(2)]
    return dict(w=w, g=[n(MH, std=0.1, mean=1.0) for _ in range(2)], b=n(MH, std=0.1),
                p=[n(MH, std=0.1, mean=1.0) for _ in range(2)]), n(MT, MH)


@pytest.mark.parametrize("tokens", [1, 5, MT])
def test_serving_step(tokens):
    d, X = _serve_params()
    m = _Serve()
    keep = m.step(X[:tokens].clone(), d)
    torch.cuda.synchronize()
    none = dict(res_scale=None, gate=None, beta_post=None)
    for i, (x_in, xn, out, par, got) in enumerate(keep):
        tm._check([t.cpu() for t in (xn, *d["w"][i])], MK, "swiglu", True, out)
        tj._forward_checks({**none, **par, "X": x_in, "Y": out[0]}, "rms",
                           "none" if i else "layer", BF, got)
        assert mlpb.mlpb_moe_last_device_error(m.moe[i].handle) == 0


def test_serving_step_captured():
    """Captured once and replayed for new tokens, as a decoding loop would."""
    d, X = _serve_params()
    m = _Serve()
    want = []
    for s in range(3):
        x = (X[s:s + 4] * (1 + s)).contiguous()
        want.append(x)
        m.step(x, d)
    x = torch.zeros(4, MH, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step(x, d)
    for s in range(3):
        x.copy_((X[s:s + 4] * (1 + s)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want[s])
    del graph


def test_calls_on_a_given_stream():
    """stream= as an object and as a handle: what a call allocates belongs to that stream, and a
    new handle serves a stream that does not wait for the default one."""
    d, X = _serve_params()
    d["g"].append(torch.ones(MH, dtype=BF, device="cuda"))
    torch.cuda.synchronize()
    z = torch.randn(64, 512, device="cuda").to(BF)
    plan = mlpb.Join(MT, MH, "rms", "rms")
    ck = mlpb.ActCheckpoint8(64, 512)
    par = dict(gamma_post=d["g"][0], gamma_pre=d["g"][1])

    def run(**kw):
        moe = mlpb.MoEDecode(MT, MH, MF, ME, MK)
        out = moe.forward(X, *d["w"][0], **kw)
        o = plan.forward(X, out[0], **par, **kw)
        g = plan.backward(None, out[0], o[0], o[2], X, X, **par, **kw)
        a = ck.save(z, **kw)
        return [*out, *o, g["dX"], g["dY"], g["dgamma_pre"], a, *ck.grad(a, **kw)], moe
    want, keep = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for kw in (dict(stream=side), dict(stream=side.cuda_stream)):
        got, m = run(**kw)
        side.synchronize()
        assert mlpb.mlpb_moe_last_device_error(m.handle, side) == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
