"""Cases of the operators around the MLP block: the join between two blocks (norms, gate,
residual scale), activation checkpoints in 8 bits, and a mixture-of-experts layer for a few
tokens.  With ``own`` false, run() is their plain form in elementary torch operations; with
``own`` true, the calls that a user makes of this repository's package."""
import math

import torch

own = False

DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-5
BLOCK = 32  # features that share one scale of an 8-bit checkpoint


# ------------------------------------------------------------------ the cases
def _join(name, op, tokens, hidden, post, pre, groups, res, x32, y32):
    return dict(name=name, op=op, tokens=tokens, hidden=hidden, post=post, pre=pre, groups=groups,
                res=res, x32=x32, y32=y32)


def _act8(name, op, tokens, ffn, tp, act):
    return dict(name=name, op=op, tokens=tokens, ffn=ffn, tp=tp, act=act)


def _moe(name, tokens, hidden, ffn, experts, topk, act, norm):
    return dict(name=name, op="moe", tokens=tokens, hidden=hidden, ffn=ffn, experts=experts,
                topk=topk, act=act, norm=norm)


def listed():
    return [
        # one decoding step of four sequences: latency
        _join("join_fwd_decode", "join_fwd", 4, 4096, "rms", "rms", 1, False, False, False),
        # a training step's tokens at the widest hidden size of the workloads
        _join("join_fwd_train", "join_fwd", 8192, 8192, "rms", "rms", 1, False, False, False),
        # eight conditioned sequences of 125 rows, a stream kept in 32 bits, LayerNorms
        _join("join_fwd_groups_f32", "join_fwd", 1000, 5120, "layer", "layer", 8, True, True, True),
        # its backward passes: the bf16 training step, and the 32-bit stream with a learned scale
        _join("join_bwd_train", "join_bwd", 8192, 8192, "rms", "rms", 1, False, False, False),
        _join("join_bwd_groups_f32", "join_bwd", 16384, 4096, "layer", "layer", 16, True, True, True),
        # fc1's output of the GELU workload, saved and used: forward and backward
        _act8("act8_step_gelu", "act8_step", 8192, 20480, 8, "gelu"),
        # the backward of the SwiGLU workload (shards of 1376 features)
        _act8("act8_grad_swiglu", "act8_grad", 16384, 11008, 8, "swiglu"),
        # a small ragged one: 77 rows, shards of 344 features (the last block of each is short)
        _act8("act8_step_ragged", "act8_step", 77, 1032, 3, "swiglu"),
        # one token through eight of 64 experts: the smallest decoding step
        _moe("moe_one_token", 1, 4096, 1376, 64, 8, "swiglu", True),
        # seven sequences, few large GELU experts
        _moe("moe_seven_gelu", 7, 5120, 2560, 16, 2, "gelu", False),
        # a batch of sixteen over many small experts
        _moe("moe_sixteen", 16, 4096, 688, 128, 8, "swiglu", True),
        # the most tokens that the decoding form takes
        _moe("moe_sixty_four", 64, 5120, 2560, 32, 4, "swiglu", True),
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    kind = rng.choice(["join_fwd", "join_bwd", "act8_step", "act8_grad", "moe", "moe"])
    if kind.startswith("join"):
        hidden = _log(rng, 64, 16384, 8)
        tokens = _log(rng, 1, min(16384, (1 << 26) // hidden))
        divisors = [g for g in range(1, tokens + 1) if tokens % g == 0]
        post, pre = rng.choice(["none", "layer", "rms"]), rng.choice(["none", "layer", "rms"])
        groups = rng.choice([0, 1, rng.choice(divisors)])
        return dict(op=kind, tokens=tokens, hidden=hidden, post=post, pre=pre, groups=groups,
                    res=rng.random() < 0.5, x32=rng.random() < 0.4, y32=rng.random() < 0.4)
    if kind.startswith("act8"):
        act = rng.choice(["gelu", "swiglu"])
        tp = rng.choice([1, 2, 3, 4, 8])
        ffn = tp * _log(rng, 8, 28672 // tp, 8)
        return dict(op=kind, tokens=_log(rng, 1, min(16384, (1 << 26) // ffn)), ffn=ffn, tp=tp,
                    act=act)
    hidden, ffn = _log(rng, 256, 8192, 64), _log(rng, 64, 4096, 8)
    most = 2 * 32 * 5120 * 2560 // (hidden * ffn)  # no more weights than the largest listed case
    experts = _log(rng, 2, max(2, min(256, most // 2)))
    return dict(op="moe", tokens=_log(rng, 1, 64), hidden=hidden, ffn=ffn, experts=experts,
                topk=min(experts, rng.randint(1, 8)), act=rng.choice(["gelu", "swiglu"]),
                norm=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, mean=0.0, dtype=BF):
    x = torch.randn(shape, generator=g, device=DEV, dtype=F32 if dtype == F32 else BF)
    if std != 1.0:
        x *= std
    if mean:
        x += mean
    return x.to(dtype)


def _segments(case):
    """Runs of features of one row of Z that start a new 8-bit block: all F of them for GELU,
    each shard's gate and up features for SwiGLU."""
    gated = case["act"] == "swiglu"
    return (2 * case["tp"], case["ffn"] // case["tp"]) if gated else (1, case["ffn"])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"].startswith("join"):
        T, H, G = case["tokens"], case["hidden"], case["groups"]
        xt, yt = F32 if case["x32"] else BF, F32 if case["y32"] else BF
        # a residual stream: wider than a block's output, a few channels far wider still
        wide = torch.ones(H, device=DEV)
        wide[:: max(1, H // 4)] = 8.0
        s["X"] = (_randn(g, T, H, dtype=F32) * 2.0 * wide).to(xt)
        s["Y"] = _randn(g, T, H, mean=0.1, dtype=F32).to(yt)
        for k in ("post", "pre"):
            on, ln = case[k] != "none", case[k] == "layer"
            s["gamma_" + k] = _randn(g, H, std=0.1, mean=1.0) if on else None
            s["beta_" + k] = _randn(g, H, std=0.02) if ln else None
        s["gate"] = _randn(g, G, H, std=0.3, mean=0.5) if G else None
        s["alpha"] = torch.full((1,), 0.8, device=DEV) if case["res"] else None
        if case["op"] == "join_bwd":
            fwd = _join_fwd_plain(s)
            s["Xout"], s["stats"] = fwd["Xout"], fwd["stats"]
            # the stream's gradient leans on the stream (it does where a loss has a say in its scale)
            s["dXout"] = (_randn(g, T, H, dtype=F32) + 0.1 * s["X"].float()).to(xt)
            s["dXn"] = _randn(g, T, H, dtype=F32).to(yt) if case["pre"] != "none" else None
        if own:
            import megatron_tensor_transformer_tma_gb300 as m
            s["plan"] = m.Join(T, H, post_norm=case["post"], pre_norm=case["pre"], gate_groups=G,
                               eps=EPS, stream_dtype=xt, block_dtype=yt, device=DEV)
    elif case["op"].startswith("act8"):
        T, F = case["tokens"], case["ffn"]
        F1 = 2 * F if case["act"] == "swiglu" else F
        Z = _randn(g, T, F1, std=1.3)
        dA = _randn(g, T, F, std=0.5)
        if case["op"] == "act8_grad":
            s["codes"], s["scales"] = _act8_quantize_plain(Z, *_segments(case))
        else:
            s["Z"] = Z
        s["dA"] = dA
        if own:
            import megatron_tensor_transformer_tma_gb300 as m
            s["plan"] = m.ActCheckpoint8(T, F, case["tp"], case["act"], device=DEV)
    else:
        T, H, Fe, E = case["tokens"], case["hidden"], case["ffn"], case["experts"]
        s["X"] = _randn(g, T, H)
        s["Wr"] = _randn(g, E, H, std=1.0 / math.sqrt(H))
        s["W1"] = _randn(g, *((E, 2, Fe, H) if case["act"] == "swiglu" else (E, Fe, H)),
                         std=1.0 / math.sqrt(H))
        s["W2"] = _randn(g, E, H, Fe, std=1.0 / math.sqrt(Fe))
        if own:
            import megatron_tensor_transformer_tma_gb300 as m
            s["plan"] = m.MoEDecode(T, H, Fe, E, case["topk"], case["act"],
                                    normalize=case["norm"], device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _norm_plain(x, kind):
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)
    return d * rstd, mean, rstd


def _rows_of(v, T):
    """[G][H] as one row for each of T tokens: group g is the g-th run of T/G rows."""
    return v.float().repeat_interleave(T // v.shape[0], 0) if v.shape[0] > 1 else v.float()


def _join_fwd_plain(s):
    T = s["tokens"]
    X, P = s["X"].float(), s["Y"].float()
    zero = torch.zeros(T, 1, device=X.device)
    mean_y = rstd_y = mean_h = rstd_h = zero
    if s["post"] != "none":
        P, mean_y, rstd_y = _norm_plain(P, s["post"])
        P = P * s["gamma_post"].float()
        if s["beta_post"] is not None:
            P = P + s["beta_post"].float()
    if s["gate"] is not None:
        P = _rows_of(s["gate"], T) * P
    Xout = ((X if s["alpha"] is None else s["alpha"] * X) + P).to(s["X"].dtype)
    out = dict(Xout=Xout)
    if s["pre"] != "none":  # of the stream as it is stored: what the backward pass will read
        Xn, mean_h, rstd_h = _norm_plain(Xout.float(), s["pre"])
        Xn = Xn * s["gamma_pre"].float()
        if s["beta_pre"] is not None:
            Xn = Xn + s["beta_pre"].float()
        out["Xn"] = Xn.to(BF)
    out["stats"] = torch.cat([mean_y, rstd_y, mean_h, rstd_h], 1)
    return out


def _norm_grad_plain(u, xh, rstd, kind):
    du = u - xh * (u * xh).mean(-1, keepdim=True)
    if kind == "layer":
        du = du - u.mean(-1, keepdim=True)
    return rstd * du


def _join_bwd_plain(s):
    T, H = s["tokens"], s["hidden"]
    mean_y, rstd_y, mean_h, rstd_h = (s["stats"][:, i:i + 1] for i in range(4))
    out = {}
    dh = s["dXout"].float()
    if s["pre"] != "none":
        hh = (s["Xout"].float() - mean_h) * rstd_h
        dXn = s["dXn"].float()
        dh = dh + _norm_grad_plain(dXn * s["gamma_pre"].float(), hh, rstd_h, s["pre"])
        out["dgamma_pre"] = (dXn * hh).sum(0)
        if s["beta_pre"] is not None:
            out["dbeta_pre"] = dXn.sum(0)
    dX = dh
    if s["alpha"] is not None:
        dX = s["alpha"] * dh
        out["dres_scale"] = (dh * s["X"].float()).sum(1).double().sum().float().reshape(1)
    out["dX"] = dX.to(s["X"].dtype)
    y = s["Y"].float()
    yh = (y - mean_y) * rstd_y if s["post"] != "none" else y
    dP = dh
    if s["gate"] is not None:
        P = yh
        if s["post"] != "none":
            P = P * s["gamma_post"].float()
            if s["beta_post"] is not None:
                P = P + s["beta_post"].float()
        out["dgate"] = (dh * P).view(s["groups"], -1, H).sum(1)
        dP = _rows_of(s["gate"], T) * dh
    if s["post"] != "none":
        out["dgamma_post"] = (dP * yh).sum(0)
        if s["beta_post"] is not None:
            out["dbeta_post"] = dP.sum(0)
        dP = _norm_grad_plain(dP * s["gamma_post"].float(), yh, rstd_y, s["post"])
    out["dY"] = dP.to(BF)
    return out


def _blocks(x, segments, width):
    """[T][segments * width] as [T][segments][blocks][32], the last block of a segment filled
    up with zeros."""
    x = x.view(-1, segments, width)
    pad = -width % BLOCK
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], segments, pad)], -1)
    return x.view(x.shape[0], segments, -1, BLOCK)


def _act8_quantize_plain(Z, segments, width):
    z = _blocks(Z.float(), segments, width)
    amax = z.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1;  127 = (127/128) 2^7
    k = torch.where(m <= 127.0 / 128.0, 7 - e, 6 - e)
    k = torch.where(amax > 0, k, torch.zeros_like(k)).clamp(max=126)
    codes = torch.round(torch.ldexp(z, k)).to(torch.int8)
    codes = codes.view(z.shape[0], segments, -1)[..., :width].reshape(Z.shape)
    return codes.contiguous(), (127 - k).to(torch.uint8).view(z.shape[0], -1)


def _act8_decode_plain(codes, scales, segments, width):
    c = _blocks(codes.float(), segments, width)
    e = scales.view(c.shape[0], segments, -1, 1).to(torch.int32) - 127
    z = torch.ldexp(c, e).view(c.shape[0], segments, -1)[..., :width]
    return z.reshape(codes.shape)


def _act_plain(z, case):
    """act(Z) of [T][F1] values in 32 bits."""
    if case["act"] == "gelu":
        u = 0.7978845608028654 * (z + 0.044715 * z * z * z)
        return z / (1.0 + torch.exp(-2.0 * u))
    gu = z.view(z.shape[0], case["tp"], 2, -1)
    a = gu[:, :, 0] / (1.0 + torch.exp(-gu[:, :, 0])) * gu[:, :, 1]
    return a.reshape(z.shape[0], -1)


def _act_grad_plain(dA, z, case):
    if case["act"] == "gelu":
        s = 1.0 / (1.0 + torch.exp(-2.0 * 0.7978845608028654 * (z + 0.044715 * z * z * z)))
        return dA * (s + z * s * (1.0 - s) * 2.0 * 0.7978845608028654
                     * (1.0 + 3.0 * 0.044715 * z * z))
    gu = z.view(z.shape[0], case["tp"], 2, -1)
    g, u = gu[:, :, 0], gu[:, :, 1]
    d = dA.view(z.shape[0], case["tp"], -1)
    s = 1.0 / (1.0 + torch.exp(-g))
    return torch.stack([d * u * s * (1.0 + g * (1.0 - s)), d * g * s], 2).reshape(z.shape)


def _act8_plain(s):
    out = {}
    if s["op"] == "act8_step":
        codes, scales = _act8_quantize_plain(s["Z"], *_segments(s))
        out["A"] = _act_plain(s["Z"].float(), s).to(BF)
    else:
        codes, scales = s["codes"], s["scales"]
    z = _act8_decode_plain(codes, scales, *_segments(s))
    out["dZ"] = _act_grad_plain(s["dA"].float(), z, s).to(BF)
    out["A_again"] = _act_plain(z, s).to(BF)
    return out


def _moe_plain(s):
    T, H, E, K = s["tokens"], s["hidden"], s["experts"], s["topk"]
    logits = s["X"].double() @ s["Wr"].double().t()  # in 64 bits: the ranks hang on small gaps
    ids = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :K]
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    w = torch.gather(p, 1, ids)
    if s["norm"]:
        w = w / w.sum(-1, keepdim=True)
    w = w.float()
    gated = s["act"] == "swiglu"
    case = dict(act=s["act"], tp=1)
    if T * K <= E:  # each pair's own expert
        W1, W2 = s["W1"][ids.reshape(-1)].float(), s["W2"][ids.reshape(-1)].float()
        x = s["X"].float().repeat_interleave(K, 0).unsqueeze(-1)
        z = torch.matmul(W1.view(T * K, -1, H), x).squeeze(-1)
        a = _act_plain(z, case)
        y = torch.matmul(W2, a.unsqueeze(-1)).view(T, K, H)
        Y = (w.unsqueeze(-1) * y).sum(1)
    else:  # every expert on every token, the ones not taken with weight zero
        comb = torch.zeros(T, E, device=w.device).scatter_(1, ids, w)
        z = torch.matmul(s["W1"].float().view(E, -1, H), s["X"].float().t())  # [E][F1][T]
        z = z.transpose(1, 2).reshape(E * T, -1)
        a = _act_plain(z, case).view(E, T, -1) * comb.t().unsqueeze(-1)
        Y = torch.matmul(a, s["W2"].float().transpose(1, 2)).sum(0)
    return dict(Y=Y.to(BF), ids=ids.to(torch.int32), weights=w)


# ------------------------------------------------------------------ one pass
def run(s):
    if not own:
        if s["op"] == "join_fwd":
            return _join_fwd_plain(s)
        if s["op"] == "join_bwd":
            return _join_bwd_plain(s)
        if s["op"] == "moe":
            return _moe_plain(s)
        return _act8_plain(s)
    plan = s["plan"]
    if s["op"] == "join_fwd":
        Xout, Xn, stats = plan.forward(s["X"], s["Y"], res_scale=s["alpha"], gate=s["gate"],
                                       gamma_post=s["gamma_post"], beta_post=s["beta_post"],
                                       gamma_pre=s["gamma_pre"], beta_pre=s["beta_pre"])
        out = dict(Xout=Xout, stats=stats)
        if Xn is not None:
            out["Xn"] = Xn
        return out
    if s["op"] == "join_bwd":
        g = plan.backward(s["X"], s["Y"], s["Xout"], s["stats"], s["dXout"], s["dXn"],
                          res_scale=s["alpha"], gate=s["gate"], gamma_post=s["gamma_post"],
                          beta_post=s["beta_post"], gamma_pre=s["gamma_pre"],
                          beta_pre=s["beta_pre"])
        return {k: v for k, v in g.items() if v is not None}
    if s["op"] == "moe":
        Y, ids, w = plan.forward(s["X"], s["Wr"], s["W1"], s["W2"])
        return dict(Y=Y, ids=ids, weights=w)
    out = {}
    if s["op"] == "act8_step":
        out["A"] = plan.save(s["Z"])
        out["dZ"], out["A_again"] = plan.grad(s["dA"])
    else:
        out["dZ"], out["A_again"] = plan.grad(s["dA"], codes=s["codes"], scales=s["scales"])
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"].startswith("join"):
        T, H, G = case["tokens"], case["hidden"], case["groups"]
        n, x, y = T * H, 4 if case["x32"] else 2, 4 if case["y32"] else 2
        pre, post = case["pre"] != "none", case["post"] != "none"
        params = 2 * H * (pre + post + (case["pre"] == "layer") + (case["post"] == "layer") + G)
        if case["op"] == "join_fwd":
            return dict(bytes=n * (x + y + x + (2 if pre else 0)) + 16 * T + params,
                        flops=n * 15.0)
        reads = n * (x + (y if post or G else 0) + (x + y if pre else 0) + (x if case["res"] else 0))
        return dict(bytes=reads + n * (x + 2) + 16 * T + 3 * params, flops=n * 30.0)
    if case["op"].startswith("act8"):
        T, F = case["tokens"], case["ffn"]
        segments, width = _segments(case)
        f1 = segments * width
        saved = f1 + segments * (-(-width // BLOCK))
        grad = T * (2 * F + saved + 2 * f1 + 2 * F)
        save = T * (2 * f1 + 2 * F + saved) if case["op"] == "act8_step" else 0
        return dict(bytes=grad + save, flops=T * F * (60.0 if save else 40.0))
    T, H, Fe, E, K = (case[k] for k in ("tokens", "hidden", "ffn", "experts", "topk"))
    mats = 3 if case["act"] == "swiglu" else 2
    # experts that T tokens reach when each takes K of E at random
    reached = E * (1.0 - (1.0 - K / E) ** T)
    return dict(bytes=reached * mats * H * Fe * 2 + E * H * 2 + 4 * T * H + 8 * T * K,
                flops=2.0 * T * K * mats * H * Fe + 2.0 * T * E * H)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _norm_exact(x, kind):
    if kind == "layer":
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    else:
        mean = torch.zeros_like(x[:, :1])
        var = torch.linalg.vector_norm(x, dim=-1, keepdim=True).square() / x.shape[1]
    return mean, torch.rsqrt(var + EPS)


def _affine_exact(s, which, xh):
    out = xh * s["gamma_" + which].double()
    return out if s["beta_" + which] is None else out + s["beta_" + which].double()


def _join_exact(s):
    T, H, G = s["tokens"], s["hidden"], s["groups"]
    alpha = 1.0 if s["alpha"] is None else s["alpha"].double()
    X, Y = s["X"].double(), s["Y"].double()
    gate = torch.ones(1, 1, H, dtype=F64, device=X.device) if G == 0 else s["gate"].double()[:, None]
    in_groups = (max(G, 1), -1, H)
    if s["op"] == "join_fwd":
        z = torch.zeros(T, 1, dtype=F64, device=X.device)
        stats, P = [z, z, z, z], Y
        if s["post"] != "none":
            stats[:2] = _norm_exact(Y, s["post"])
            P = _affine_exact(s, "post", (Y - stats[0]) * stats[1])
        h = alpha * X + (P.view(in_groups) * gate).view(T, H)
        out = dict(Xout=h)
        if s["pre"] != "none":
            stats[2:] = _norm_exact(h, s["pre"])
            out["Xn"] = _affine_exact(s, "pre", (h - stats[2]) * stats[3])
        # the norm reads the stored stream: where that is bf16 its statistics are not h's own
        out["stats"] = torch.cat(stats, 1) if s["x32"] or s["pre"] == "none" else None
        return out
    st = s["stats"].double()
    out = dict.fromkeys(("dgamma_pre", "dbeta_pre", "dres_scale", "dgate", "dgamma_post",
                         "dbeta_post"))
    total = s["dXout"].double()
    if s["pre"] != "none":
        r = st[:, 3:4]
        xh = (s["Xout"].double() - st[:, 2:3]) * r
        d = s["dXn"].double()
        w = d * s["gamma_pre"].double()
        along = torch.einsum("th,th->t", w, xh)[:, None] / H
        flat = w.sum(-1, keepdim=True) / H if s["pre"] == "layer" else 0.0
        total = total + r * (w - flat - xh * along)
        out["dgamma_pre"] = torch.einsum("th,th->h", d, xh)
        out["dbeta_pre"] = d.sum(0) if s["pre"] == "layer" else None
    out["dX"] = alpha * total
    if s["alpha"] is not None:
        out["dres_scale"] = torch.einsum("th,th->", total, X).reshape(1)
    yh = (Y - st[:, 0:1]) * st[:, 1:2] if s["post"] != "none" else Y
    s0 = total.view(in_groups).sum(1)
    s1 = torch.einsum("grh,grh->gh", total.view(in_groups), yh.reshape(in_groups))
    if G:
        out["dgate"] = s1 if s["post"] == "none" else _affine_exact(s, "post", s1) if \
            s["beta_post"] is None else s1 * s["gamma_post"].double() + s0 * s["beta_post"].double()
    dP = (total.view(in_groups) * gate).view(T, H)
    if s["post"] != "none":
        out["dgamma_post"] = (gate[:, 0] * s1).sum(0)
        out["dbeta_post"] = (gate[:, 0] * s0).sum(0) if s["post"] == "layer" else None
        w = dP * s["gamma_post"].double()
        along = torch.einsum("th,th->t", w, yh)[:, None] / H
        flat = w.sum(-1, keepdim=True) / H if s["post"] == "layer" else 0.0
        dP = st[:, 1:2] * (w - flat - yh * along)
    out["dY"] = dP
    return {k: v for k, v in out.items() if v is not None}


def _act_exact(z, s):
    if s["act"] == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    g, u = z.unflatten(1, (s["tp"], 2, -1)).unbind(2)
    return (g * torch.sigmoid(g) * u).flatten(1)


def _act_slope_exact(z, d, s):
    if s["act"] == "gelu":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z ** 3))
        return d * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 0.134145 * z * z))
    g, u = z.unflatten(1, (s["tp"], 2, -1)).unbind(2)
    d = d.unflatten(1, (s["tp"], -1))
    sg = torch.sigmoid(g)
    return torch.stack([d * u * (sg + g * sg * (1.0 - sg)), d * g * sg], 2).flatten(1)


def _act8_decoded_exact(s):
    """The values that the 8-bit checkpoint of each block stands for."""
    segments, width = _segments(s)
    out = torch.empty(s["tokens"], segments, width, dtype=F64, device=DEV)
    for b0 in range(0, width, BLOCK):
        b1 = min(width, b0 + BLOCK)
        if s["op"] == "act8_step":
            z = s["Z"].view(out.shape)[..., b0:b1].double()
            top = z.abs().amax(-1, keepdim=True)
            k = torch.floor(torch.log2(127.0 / top.clamp(min=1e-300)))
            # log2 may be off at a border: settle it by the inequality itself
            k = torch.where(top * torch.exp2(k) > 127.0, k - 1, k)
            k = torch.where(top * torch.exp2(k + 1) <= 127.0, k + 1, k).clamp(max=126)
            step = torch.exp2(-torch.where(top > 0, k, torch.zeros_like(k)))
            out[..., b0:b1] = torch.round(z / step) * step
        else:
            e = s["scales"].view(s["tokens"], segments, -1)[..., b0 // BLOCK, None].double()
            out[..., b0:b1] = s["codes"].view(out.shape)[..., b0:b1].double() * torch.exp2(e - 127.0)
    return out.flatten(1)


def _act8_exact(s):
    out = {}
    if s["op"] == "act8_step":
        out["A"] = _act_exact(s["Z"].double(), s)
    z = _act8_decoded_exact(s)
    out["dZ"] = _act_slope_exact(z, s["dA"].double(), s)
    out["A_again"] = _act_exact(z, s)
    return out


def _moe_exact(s):
    K, E = s["topk"], s["experts"]
    p = torch.softmax(torch.einsum("th,eh->te", s["X"].double(), s["Wr"].double()), -1)
    w, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    w, ids = w[:, :K], ids[:, :K]
    if s["norm"]:
        w = w / w.sum(-1, keepdim=True)
    Y = torch.zeros(s["tokens"], s["hidden"], dtype=F64, device=DEV)
    for e in range(E):
        rows, slot = (ids == e).nonzero(as_tuple=True)
        if rows.numel():
            z = s["X"][rows].double() @ s["W1"][e].double().flatten(0, -2).t()
            a = _act_exact(z, dict(act=s["act"], tp=1))
            Y.index_add_(0, rows, w[rows, slot, None] * (a @ s["W2"][e].double().t()))
    return dict(Y=Y, ids=None, weights=w)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("join"):
        return _join_exact(s)
    return _moe_exact(s) if case["op"] == "moe" else _act8_exact(s)
