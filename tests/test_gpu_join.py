"""GPU parity of the join between two blocks against its fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24).  A row's sum adds at most 16 values in a thread,
then 5 shuffles, then up to 32 warps: 53 roundings, so a mean is within 53 u of the mean of
magnitudes, and 1/sqrt(mean square + eps) within 33 u of its value.  A normalised value is
within 64 u of (|x| + |mean| + mean|x|) rs, its "magnitude".  The backward multiplies three such
factors (the sum g xh, xh, rs): 200 u of the magnitudes of the terms; dY chains two of them:
400 u.  Sums over rows add at most T more roundings: (400 + T) u of the sum of magnitudes.
bf16 outputs add half a step of their value, 2^-8 at most.  Xn and its statistics are compared
with the norm of the stream that the GPU stored, which is how they are defined.
"""
import threading

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb
from oracle import join

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def _make(T, H, post, pre, G, res, xt, yt, seed=0, dev="cuda"):
    g = torch.Generator().manual_seed(1000 * T + H + seed)

    def n(*shape, std=1.0, mean=0.0, dtype=BF):
        return (torch.randn(shape, generator=g) * std + mean).to(dtype).to(dev)
    wide = torch.ones(H)
    wide[::7] = 8.0
    d = dict(X=(torch.randn(T, H, generator=g) * 2 * wide).to(xt).to(dev),
             Y=n(T, H, mean=0.5, dtype=yt),
             res_scale=torch.full((1,), 0.8, device=dev) if res else None,
             gate=n(G, H, std=0.3, mean=0.5) if G else None)
    for k, kind in (("post", post), ("pre", pre)):
        d["gamma_" + k] = n(H, std=0.1, mean=1.0) if kind != "none" else None
        d["beta_" + k] = n(H, std=0.2) if kind == "layer" else None
    d["dXout"] = n(T, H, dtype=xt)
    d["dXn"] = n(T, H, dtype=yt) if pre != "none" else None
    return d


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _check(name, got, ref, tol, bf16=False):
    got = _f64(got)
    bound = tol + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0) + 1e-30
    assert got.shape == ref.shape, name
    assert (np.abs(got - ref) <= bound).all(), (
        name, float((np.abs(got - ref) - bound).max()), float(np.abs(ref).max()))


def _mag(x, rs_stats, kind):
    """Magnitude of a normalised row: (|x| + |mean| + mean|x|) / sqrt(...)."""
    if kind == "none":
        return np.abs(x)
    _, mu, rs = rs_stats
    return (np.abs(x) + np.abs(mu) + np.abs(x).mean(1, keepdims=True)) * rs


def _abs_affine(m, kind, gamma, beta):
    if kind == "none":
        return m
    return m * np.abs(gamma) + (np.abs(beta) if kind == "layer" else 0.0)


def _forward_checks(d, post, pre, xt, out):
    f = {k: _f64(v) for k, v in d.items()}
    T = f["X"].shape[0]
    alpha = 1.0 if f["res_scale"] is None else float(f["res_scale"][0])
    Xout, Xn, stats = out
    ref = join.forward(f["X"], f["Y"], alpha, f["gate"], post, f["gamma_post"], f["beta_post"],
                       "none", None, None, EPS)
    ystat = join.norm(f["Y"], post, EPS)
    p_mag = _abs_affine(_mag(f["Y"], ystat, post), post, f["gamma_post"], f["beta_post"])
    terms = abs(alpha) * np.abs(f["X"]) + np.abs(join.gate_rows(f["gate"], T)) * p_mag
    _check("Xout", Xout, ref["Xout"], 64 * U * terms, xt == BF)
    h = _f64(Xout)
    hstat = join.norm(h, pre, EPS)
    st = _f64(stats)
    for i, (x, s, kind) in enumerate(((f["Y"], ystat, post), (h, hstat, pre))):
        if kind == "none":
            assert (st[:, 2 * i:2 * i + 2] == 0).all()
            continue
        _check("mean", stats[:, 2 * i:2 * i + 1], s[1], 53 * U * np.abs(x).mean(1, keepdims=True))
        _check("rstd", stats[:, 2 * i + 1:2 * i + 2], s[2], 33 * U * s[2])
    if pre == "none":
        assert Xn is None
        return
    mag = _abs_affine(_mag(h, hstat, pre), pre, f["gamma_pre"], f["beta_pre"])
    want = hstat[0] * f["gamma_pre"] + (f["beta_pre"] if pre == "layer" else 0.0)
    _check("Xn", Xn, want, 64 * U * mag, True)


def _backward_checks(d, post, pre, xt, Xout, got, base=None):
    f = {k: _f64(v) for k, v in d.items()}
    T, H = f["dXout"].shape if f["dXout"] is not None else f["X"].shape
    alpha = 1.0 if f["res_scale"] is None else float(f["res_scale"][0])
    h = _f64(Xout)
    ref = join.backward(f["X"], f["Y"], h, alpha, f["gate"], post, f["gamma_post"],
                        f["beta_post"], pre, f["gamma_pre"], EPS, f["dXout"], f["dXn"])
    dh = np.zeros((T, H)) if f["dXout"] is None else np.abs(f["dXout"])
    if pre != "none":
        s = join.norm(h, pre, EPS)
        mag = _mag(h, s, pre)
        g = np.abs(f["dXn"] * f["gamma_pre"])
        dh = dh + s[2] * (g + g.mean(1, keepdims=True) + mag * (g * mag).mean(1, keepdims=True))
        sums = {"dgamma_pre": (np.abs(f["dXn"]) * mag).sum(0)}
        if pre == "layer":
            sums["dbeta_pre"] = np.abs(f["dXn"]).sum(0)
    else:
        sums = {}
    _check("dX", got["dX"], ref["dX"], 200 * U * abs(alpha) * dh, xt == BF)
    if f["res_scale"] is not None:
        sums["dres_scale"] = np.array([(dh * np.abs(f["X"])).sum()])
    s = join.norm(f["Y"], post, EPS)
    mag = _mag(f["Y"], s, post)
    gate = np.abs(join.gate_rows(f["gate"], T))
    dP = gate * dh
    if f["gate"] is not None:
        P = _abs_affine(mag, post, f["gamma_post"], f["beta_post"])
        sums["dgate"] = (dh * P).reshape(f["gate"].shape[0], -1, H).sum(1)
    if post != "none":
        sums["dgamma_post"] = (dP * mag).sum(0)
        if post == "layer":
            sums["dbeta_post"] = dP.sum(0)
        t = dP * np.abs(f["gamma_post"])
        dP = s[2] * (t + t.mean(1, keepdims=True) + mag * (t * mag).mean(1, keepdims=True))
    _check("dY", got["dY"], ref["dY"], 400 * U * dP, True)
    for k in ("dres_scale", "dgate", "dgamma_post", "dbeta_post", "dgamma_pre", "dbeta_pre"):
        if k not in sums:
            assert got[k] is None, k
            continue
        want = ref[k] + (0.0 if base is None else base)
        _check(k, got[k], want, (400 + T) * U * (sums[k] + (0.0 if base is None else abs(base))))


def _run(T, H, post, pre, G, res, xt, yt, seed=0):
    d = _make(T, H, post, pre, G, res, xt, yt, seed)
    plan = mlpb.Join(T, H, post, pre, G, EPS, xt, yt)
    keys = ("res_scale", "gate", "gamma_post", "beta_post", "gamma_pre", "beta_pre")
    par = {k: d[k] for k in keys}
    out = plan.forward(d["X"], d["Y"], **par)
    _forward_checks(d, post, pre, xt, out)
    got = plan.backward(d["X"], d["Y"], out[0], out[2], d["dXout"], d["dXn"], **par)
    _backward_checks(d, post, pre, xt, out[0], got)
    return d, par, plan, out, got


KINDS = ["none", "layer", "rms"]


@pytest.mark.parametrize("post", KINDS)
@pytest.mark.parametrize("pre", KINDS)
@pytest.mark.parametrize("G", [0, 1, 5])
def test_every_norm_and_gate(post, pre, G):
    _run(35, 264, post, pre, G, G != 0, BF, BF)
    _run(35, 264, post, pre, G, G == 0, F32, F32)


# one row and many, a row per warp up to a row per 1024 threads, ragged widths, several rows a
# thread group, more groups than CTAs
SHAPES = [(1, 8), (1, 4096), (4, 4096), (3, 64), (700, 72), (130, 520), (61, 1032), (257, 1496),
          (350, 2056), (700, 4096), (331, 8192), (5, 8200), (190, 16384)]


@pytest.mark.parametrize("T,H", SHAPES)
def test_shapes_and_types(T, H):
    i = SHAPES.index((T, H))
    types = [(BF, BF), (F32, F32), (BF, F32), (F32, BF)]
    _run(T, H, "rms", "rms", 1, False, *types[i % 4])
    _run(T, H, "layer", "layer", T, True, *types[(i + 1) % 4])
    _run(T, H, "layer", "rms", 0, True, *types[(i + 2) % 4])


# widths that leave warps, or CTAs of a row, with few columns or none; rows that share a CTA
@pytest.mark.parametrize("H", [256, 264, 512, 776, 1536, 2184, 2936, 4392, 6024, 6152, 7000, 8208,
                               12288, 12296, 13000, 16376])
def test_widths(H):
    for i, T in enumerate((5, 460)):
        types = [(BF, BF), (F32, F32), (BF, F32), (F32, BF)][(H // 8 + i) % 4]
        _run(T, H, "layer", "layer", 5, True, *types)
        _run(T, H, "rms", "rms", 0, False, *types)
        _run(T, H, "none", "layer", T, True, *types)


@pytest.mark.parametrize("T,H,G", [(5000, 264, 5000), (3000, 512, 1500), (2100, 1024, 2100),
                                   (2000, 2048, 1000), (700, 4392, 700), (333, 9000, 333),
                                   (1900, 72, 950), (40, 520, 40)])
def test_many_short_groups(T, H, G):
    """A gate for each token or pair: rows of a CTA in groups of their own, copies that run on from
    a group to the next, walkers without a group."""
    _run(T, H, "layer", "rms", G, True, BF, BF)
    _run(T, H, "rms", "rms", G, False, F32, F32)


def test_rows_of_two_ctas():
    """Above 8192 columns: in place, accumulated, captured, groups more and fewer than walkers."""
    for G in (2, 380):
        T, H = 380, 9000
        d, par, plan, out, got = _run(T, H, "layer", "rms", G, True, BF, BF)
        acc = mlpb.Join(T, H, "layer", "rms", G, EPS, accumulate=True)
        grads = acc.alloc_grads(True)
        grads["dX"] = d["dXout"].clone()
        stat = (out[0], out[2])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            acc.backward(d["X"], d["Y"], *stat, grads["dX"], d["dXn"], grads=grads, **par)
        graph.replay()
        torch.cuda.synchronize()
        for k, v in got.items():
            assert (v is None and grads[k] is None) or torch.equal(v, grads[k]), k
        del graph


@pytest.mark.parametrize("T,H,G", [(1000, 320, 8), (2048, 64, 1024), (1500, 136, 500),
                                   (400, 8192, 400), (640, 1024, 2)])
def test_groups(T, H, G):
    _run(T, H, "layer", "layer", G, True, BF, BF)
    _run(T, H, "none", "rms", G, False, F32, BF)


def test_same_bits_every_run_and_in_place():
    d, par, plan, out, got = _run(333, 1000, "layer", "layer", 3, True, BF, BF)
    again = plan.backward(d["X"], d["Y"], out[0], out[2], d["dXout"], d["dXn"], **par)
    for k, v in got.items():
        assert torch.equal(v, again[k]), k
    # the stream updated in place, and its gradient
    X = d["X"].clone()
    o = plan.forward(X, d["Y"], Xout=X, **par)
    assert torch.equal(o[0], out[0]) and torch.equal(o[1], out[1])
    grads = plan.alloc_grads(True)
    grads["dX"] = d["dXout"].clone()
    g = plan.backward(d["X"], d["Y"], out[0], out[2], grads["dX"], d["dXn"], grads=grads, **par)
    for k, v in got.items():
        assert torch.equal(v, g[k]), k


def test_accumulated_gradients():
    for G in (2, 700):  # a group over many CTAs, and a CTA over many groups
        T, H = 700, 520
        d = _make(T, H, "layer", "layer", G, True, BF, BF)
        plan = mlpb.Join(T, H, "layer", "layer", G, EPS, accumulate=True)
        par = {k: d[k] for k in ("res_scale", "gate", "gamma_post", "beta_post", "gamma_pre",
                                 "beta_pre")}
        out = plan.forward(d["X"], d["Y"], **par)
        grads = plan.alloc_grads(True)
        for k, v in grads.items():
            if k not in ("dX", "dY"):
                assert (v == 0).all()
                v.fill_(3.0)
        got = plan.backward(d["X"], d["Y"], out[0], out[2], d["dXout"], d["dXn"], grads=grads,
                            **par)
        _backward_checks(d, "layer", "layer", BF, out[0], got, base=3.0)


def test_without_a_stream_gradient():
    """The last join of a network: only its normalised output is used."""
    d = _make(40, 264, "rms", "layer", 1, True, BF, F32)
    plan = mlpb.Join(40, 264, "rms", "layer", 1, EPS, BF, F32)
    par = {k: d[k] for k in ("res_scale", "gate", "gamma_post", "beta_post", "gamma_pre",
                             "beta_pre")}
    out = plan.forward(d["X"], d["Y"], **par)
    d["dXout"] = None
    got = plan.backward(d["X"], d["Y"], out[0], out[2], None, d["dXn"], **par)
    _backward_checks(d, "rms", "layer", BF, out[0], got)


@pytest.mark.parametrize("pre", ["layer", "rms"])
@pytest.mark.parametrize("xt", [BF, F32])
def test_norm_alone(pre, xt):
    """Without a block: the norm in front of a first one."""
    T, H = 77, 1032
    d = _make(T, H, "none", pre, 0, False, xt, BF)
    plan = mlpb.Join(T, H, pre_norm=pre, eps=EPS, stream_dtype=xt, has_block=False)
    par = dict(gamma_pre=d["gamma_pre"], beta_pre=d["beta_pre"])
    none, Xn, stats = plan.forward(d["X"], **par)
    assert none is None
    d["Y"] = torch.zeros_like(d["X"])
    _forward_checks(d, "none", pre, xt, (d["X"], Xn, stats))
    got = plan.backward(None, None, d["X"], stats, d["dXout"], d["dXn"], **par)
    assert got["dY"] is None
    got["dY"] = got["dX"].to(BF)  # the oracle's block gradient is the stream's here
    _backward_checks(d, "none", pre, xt, d["X"], got)


def test_no_tokens():
    plan = mlpb.Join(0, 64, "layer", "layer", 1, EPS)
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    v = torch.ones(64, dtype=BF, device="cuda")
    par = dict(gate=v[None], gamma_post=v, beta_post=v, gamma_pre=v, beta_pre=v,
               res_scale=torch.ones(1, device="cuda"))
    Xout, Xn, stats = plan.forward(e, e, **par)
    assert Xout.shape == (0, 64) and stats.shape == (0, 4)
    grads = plan.alloc_grads(True)
    for k, g in grads.items():
        g.fill_(7.0)
    got = plan.backward(e, e, Xout, stats, e, e, grads=grads, **par)
    for k in ("dres_scale", "dgate", "dgamma_post", "dbeta_post", "dgamma_pre", "dbeta_pre"):
        assert (got[k] == 0).all(), k


def test_a_bad_row_stays_alone():
    """A row of NaN, one with an infinity and one of zeros leave every other row as it was."""
    T, H = 40, 520
    d = _make(T, H, "layer", "rms", 1, False, BF, BF)
    plan = mlpb.Join(T, H, "layer", "rms", 1, EPS)
    par = {k: d[k] for k in ("gate", "gamma_post", "beta_post", "gamma_pre", "beta_pre")}
    a = plan.forward(d["X"], d["Y"], **par)
    X, Y = d["X"].clone(), d["Y"].clone()
    X[3], Y[9, 7] = float("nan"), float("inf")
    X[20], Y[20] = 0.0, 0.0
    b = plan.forward(X, Y, **par)
    keep = [i for i in range(T) if i not in (3, 9, 20)]
    for s, t in zip(a, b):
        assert torch.equal(s[keep], t[keep])
        assert torch.isnan(t[3]).any() and torch.isnan(t[9]).any()
        assert torch.isfinite(t[20]).all()


def test_offset_rows_and_large_values():
    """A common offset a thousand times the spread costs a LayerNorm no digits of its variance."""
    T, H = 16, 4096
    d = _make(T, H, "layer", "layer", 0, False, F32, F32)
    d["Y"] = d["Y"] + 1000.0
    d["X"] = d["X"] * 1e3
    plan = mlpb.Join(T, H, "layer", "layer", 0, EPS, F32, F32)
    par = {k: d[k] for k in ("gamma_post", "beta_post", "gamma_pre", "beta_pre")}
    _forward_checks(d, "layer", "layer", F32, plan.forward(d["X"], d["Y"], **par))


def test_other_stream_and_two_graphs():
    d, par, plan, out, got = _run(100, 1032, "layer", "rms", 4, True, BF, BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o = plan.forward(d["X"], d["Y"], **par)
        g = plan.backward(d["X"], d["Y"], o[0], o[2], d["dXout"], d["dXn"], **par)
    s.synchronize()
    assert torch.equal(o[0], out[0]) and torch.equal(g["dgate"], got["dgate"])
    # two captured graphs of their own plans replay interleaved
    graphs = []
    for _ in range(2):
        p2 = mlpb.Join(100, 1032, "layer", "rms", 4, EPS)
        bufs = p2.forward(d["X"], d["Y"], **par)
        grads = p2.alloc_grads(True)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            p2.forward(d["X"], d["Y"], Xout=bufs[0], Xn=bufs[1], stats=bufs[2], **par)
            p2.backward(d["X"], d["Y"], bufs[0], bufs[2], d["dXout"], d["dXn"], grads=grads, **par)
        grads = {k: v for k, v in grads.items() if v is not None}
        for t in (*bufs, *grads.values()):
            t.zero_()
        graphs.append((gr, grads, p2, bufs))  # a graph needs its buffers alive
    for _ in range(2):
        for gr, *_ in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for _, grads, *_ in graphs:
        for k, v in grads.items():
            assert torch.equal(v, got[k]), k


def test_host_threads():
    """Threads with plans of different sizes for the same kernels."""
    wrong = []

    def work(T, G, res):
        with torch.cuda.stream(torch.cuda.Stream()):
            d = _make(T, 4096, "rms", "rms", G, res, BF, BF)
            plan = mlpb.Join(T, 4096, "rms", "rms", G, EPS)
            par = {k: d[k] for k in ("res_scale", "gate", "gamma_post", "gamma_pre")}
            first = None
            for i in range(60):
                o = plan.forward(d["X"], d["Y"], **par)
                g = plan.backward(d["X"], d["Y"], o[0], o[2], d["dXout"], d["dXn"], **par)
                out = [o[0], o[1], g["dX"], g["dY"], g["dgamma_pre"]]
                first = first or [t.clone() for t in out]
                if not all(torch.equal(a, b) for a, b in zip(first, out)):
                    wrong.append((T, i))
    threads = [threading.Thread(target=work, args=a)
               for a in ((4, 0, False), (1500, 1, True), (700, 0, False))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_offsets_past_32_bits():
    """Element offsets beyond 2^31: the last rows of a 4.3 GB stream."""
    T, H = 131080, 16384
    X = torch.zeros(T, H, dtype=BF, device="cuda")
    Y = torch.zeros(T, H, dtype=BF, device="cuda")
    d = _make(16, H, "rms", "rms", 1, False, BF, BF)
    X[-16:], Y[-16:] = d["X"], d["Y"]
    par = {k: d[k] for k in ("gate", "gamma_post", "gamma_pre")}
    big = mlpb.Join(T, H, "rms", "rms", 1, EPS)
    small = mlpb.Join(16, H, "rms", "rms", 1, EPS)
    a = big.forward(X, Y, **par)
    b = small.forward(d["X"], d["Y"], **par)
    for s, t in zip(a, b):
        assert torch.equal(s[-16:], t)
    dX = torch.zeros(T, H, dtype=BF, device="cuda")
    dX[-16:] = d["dXout"]
    dXn = torch.zeros(T, H, dtype=BF, device="cuda")
    dXn[-16:] = d["dXn"]
    ga = big.backward(None, Y, a[0], a[2], dX, dXn, **par)
    gb = small.backward(None, d["Y"], b[0], b[2], d["dXout"], d["dXn"], **par)
    assert torch.equal(ga["dX"][-16:], gb["dX"]) and torch.equal(ga["dY"][-16:], gb["dY"])
    assert torch.allclose(ga["dgamma_pre"], gb["dgamma_pre"], rtol=1e-5, atol=1e-4)


def test_refusals():
    d = _make(4, 64, "rms", "layer", 2, True, BF, BF)
    plan = mlpb.Join(4, 64, "rms", "layer", 2, EPS)
    par = {k: d[k] for k in ("res_scale", "gate", "gamma_post", "gamma_pre", "beta_pre")}
    Xout, Xn, stats = plan.forward(d["X"], d["Y"], **par)
    for k, bad in (("gate", d["gate"][:1]), ("gamma_post", d["gamma_post"].float()),
                   ("res_scale", torch.ones(2, device="cuda")), ("gamma_pre", None),
                   ("gate", d["gate"].cpu())):
        with pytest.raises((ValueError, TypeError, mlpb.MLPBError)):
            plan.forward(d["X"], d["Y"], **{**par, k: bad})
    with pytest.raises(ValueError):
        plan.forward(d["X"].t().contiguous().t(), d["Y"], **par)
    with pytest.raises(TypeError):
        plan.forward(d["X"], d["Y"].float(), **par)
    with pytest.raises(ValueError, match="workspace"):
        plan.workspace = plan.workspace[:128]
        plan.backward(d["X"], d["Y"], Xout, stats, d["dXout"], d["dXn"], **par)
