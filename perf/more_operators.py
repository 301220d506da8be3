"""Cases of the operators of a projection's training and serving around the MLP block: a linear
layer on 8-bit floating point with a scale for each block of 128, and the orthogonalised update
of a weight by Newton-Schulz products.  With ``own`` false, run() is their plain form in
elementary torch operations; with ``own`` true, the calls that a user makes of this repository's
package."""
import math

import torch

own = False

DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn
BLOCK = 128  # features (and, in a weight, rows too) that share one scale
COEF = (3.4445, -4.7750, 2.0315)  # a, b, c of X <- a X + (b A + c A A) X, A = X X^T
STEPS = 5
MOMENTUM = 0.95
DECAY = 0.1
LR = 1e-4


# ------------------------------------------------------------------ the cases
def _linear(name, op, tokens, inputs, outputs, accumulate=False):
    return dict(name=name, op=op, tokens=tokens, inputs=inputs, outputs=outputs,
                accumulate=accumulate)


def _ortho(name, op, batch, rows, cols, half=False):
    return dict(name=name, op=op, batch=batch, rows=rows, cols=cols, half=half)


def listed():
    return [
        # one token through the GELU workload's first projection: a decoding step, latency and
        # the weight's bytes
        _linear("linear_one_token", "linear_fwd", 1, 5120, 20480),
        # sixteen sequences through a second projection: few outputs, a long sum
        _linear("linear_sixteen", "linear_fwd", 16, 11008, 4096),
        # a short ragged prompt through a small layer whose last blocks are not full
        _linear("linear_ragged", "linear_fwd", 77, 1032, 344),
        # a training step's first projection at the GELU workload's sizes
        _linear("linear_fwd_train", "linear_fwd", 8192, 5120, 20480),
        # the backward of its second projection: gradients of the inputs and of the weight
        _linear("linear_bwd_train", "linear_bwd", 8192, 20480, 5120),
        # a ragged micro-batch added into a gradient that other micro-batches have begun
        _linear("linear_bwd_ragged", "linear_bwd", 1000, 4096, 1376, accumulate=True),
        # what a step of the SwiGLU workload does with one projection: the updated weight is laid
        # out, forward, backward
        _linear("linear_step", "linear_step", 16384, 4096, 11008),
        # the router of 64 experts: the smallest matrix that is orthogonalised
        _ortho("ortho_router", "ortho", 1, 64, 4096),
        # one shard's gate projection, from a bf16 gradient
        _ortho("ortho_shard_bf16", "ortho", 1, 1376, 4096, half=True),
        # three odd tall matrices
        _ortho("ortho_odd_tall", "ortho", 3, 1000, 333),
        # the optimiser's step of the SwiGLU workload's first weight: gate and up of eight shards
        _ortho("muon_swiglu_w1", "muon", 16, 1376, 4096),
        # and of the GELU workload's second one: eight tall shards
        _ortho("muon_gelu_w2", "muon", 8, 5120, 2560),
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_fwd", "linear_bwd", "linear_step", "ortho", "ortho",
                     "muon"])
    if op.startswith("linear"):
        inputs, outputs = _log(rng, 64, 20480, 8), _log(rng, 64, 20480, 8)
        inputs = max(64, min(inputs, 5120 * 20480 // outputs // 8 * 8))
        # serving has few rows as often as many
        most = min(16384, (1 << 39) // (inputs * outputs))
        tokens = _log(rng, 1, min(64, most)) if op == "linear_fwd" and rng.random() < 0.5 \
            else _log(rng, 1, most)
        return dict(op=op, tokens=tokens, inputs=inputs, outputs=outputs,
                    accumulate=op == "linear_bwd" and rng.random() < 0.5)
    rows, cols = _log(rng, 16, 8192), _log(rng, 16, 8192)
    cost = rows * cols * min(rows, cols)
    most = 8 * 5120 * 2560 * 2560 // cost
    if most < 1:
        cols, most = max(16, cols // 8), 1
    batch = _log(rng, 1, max(1, min(16, most, (1 << 26) // (rows * cols))))
    return dict(op=op, batch=batch, rows=rows, cols=cols,
                half=op == "ortho" and rng.random() < 0.4)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=BF):
    x = torch.randn(shape, generator=g, device=DEV, dtype=F32 if dtype == F32 else BF)
    if std != 1.0:
        x *= std
    return x.to(dtype)


def _activations(g, T, H):
    """Rows of different sizes, and a few features far wider than the rest."""
    x = torch.randn(T, H, generator=g, device=DEV, dtype=F32)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV))
    x[:, :: max(1, H // 8)] *= 20.0
    return x.to(BF)


def _gradient(g, *shape):
    """A weight's gradient: a few strong directions whose sizes fall off, and noise."""
    n, (r, c) = math.prod(shape[:-2]), shape[-2:]
    k = max(1, min(r, c) // 16)
    u = torch.randn(n, r, k, generator=g, device=DEV) / math.sqrt(k)
    v = torch.randn(n, k, c, generator=g, device=DEV)
    v *= torch.logspace(0, -1.5, k, device=DEV)[:, None]
    return 1e-3 * (torch.bmm(u, v) + 0.2 * torch.randn(n, r, c, generator=g, device=DEV))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"].startswith("linear"):
        T, K, N = case["tokens"], case["inputs"], case["outputs"]
        s["X"] = _activations(g, T, K)
        W = _randn(g, N, K, std=1.0 / math.sqrt(K))
        if case["op"] == "linear_step":
            s["W"] = W
        else:  # the weight as it is kept between updates
            s["Wq"], s["We"] = _quantize_plain(W, BLOCK)
        if case["op"] != "linear_fwd":
            s["dY"] = _randn(g, T, N, std=1e-3)
        if case["op"] == "linear_bwd":  # what the forward pass has kept of X
            s["Xq"], s["Xe"] = _quantize_plain(s["X"].t(), 1)
        if case["accumulate"]:
            s["dW"] = _randn(g, N, K, std=1e-3 * math.sqrt(T), dtype=F32)
        if own:
            import megatron_tensor_transformer_tma_gb300 as m
            s["plan"] = m.Linear8(T, K, N, training=case["op"] != "linear_fwd", device=DEV)
            if case["op"] != "linear_step":
                s["plan"].load(W)
            if case["op"] == "linear_bwd":
                s["plan"].forward(s["X"])
    else:
        shape = (case["batch"], case["rows"], case["cols"])
        s["G"] = _gradient(g, *shape).to(BF if case["half"] else F32)
        if case["op"] == "muon":
            s["M"] = 5.0 * _gradient(g, *shape) + 5.0 * s["G"]
            s["W"] = _randn(g, *shape, std=0.02, dtype=F32)
            s["lr"] = torch.full((1,), LR, device=DEV)
        if own:
            import megatron_tensor_transformer_tma_gb300 as m
            s["plan"] = m.Muon(case["rows"], case["cols"], case["batch"], steps=STEPS,
                               coefficients=COEF, momentum=MOMENTUM, nesterov=True,
                               weight_decay=DECAY, scale=_scale(case), device=DEV)
    return s


def _scale(case):
    return 0.2 * math.sqrt(max(case["rows"], case["cols"]))


# ------------------------------------------------------------------ plain forms
def _blocks(x, rows):
    """[R][C] as [ceil(R / rows)][rows][ceil(C / 128)][128], filled up with zeros."""
    R, C = x.shape
    x = torch.nn.functional.pad(x, (0, -C % BLOCK, 0, -R % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // BLOCK, BLOCK)


def _quantize_plain(x, rows):
    """E4M3 codes [R][C] and the exponents of the scales of blocks of `rows` x 128."""
    R, C = x.shape
    b = _blocks(x.float(), rows)
    amax = b.abs().amax((1, 3), keepdim=True)
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1;  448 = 0.875 2^9
    k = torch.where(m <= 0.875, 9 - e, 8 - e)
    k = torch.where(amax > 0, k, torch.zeros_like(k)).clamp(max=126)
    q = torch.ldexp(b, k).to(E4M3).view(-1, b.shape[2] * BLOCK)[:R, :C]
    return q.contiguous(), -k[:, 0, :, 0]


def _values_plain(q, e, rows):
    """What the codes stand for, in 32 bits."""
    e = e.repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return torch.ldexp(q.float(), e)


def _rounded_plain(x, rows=1):
    return _values_plain(*_quantize_plain(x, rows), rows)


def _linear_plain(s):
    out = {}
    if s["op"] == "linear_step":
        w = _rounded_plain(s["W"], BLOCK)
    else:
        w = _values_plain(s["Wq"], s["We"], BLOCK)
    if s["op"] != "linear_bwd":
        out["Y"] = torch.matmul(_rounded_plain(s["X"]), w.t()).to(BF)
    if s["op"] != "linear_fwd":
        out["dX"] = torch.matmul(_rounded_plain(s["dY"]), w).to(BF)
        xt = _rounded_plain(s["X"].t()) if s["op"] == "linear_step" \
            else _values_plain(s["Xq"], s["Xe"], 1)
        dW = torch.matmul(_rounded_plain(s["dY"].t()), xt.t())
        out["dW"] = s["dW"].add_(dW) if s["accumulate"] else dW
    return out


def _ortho_plain(u):
    """[n][r][c] with every singular value of each matrix taken through STEPS odd polynomials."""
    a, b, c = COEF
    x = u.float()
    norm = torch.sqrt((x * x).sum((1, 2), keepdim=True))
    x = x / torch.where(norm > 0, norm, torch.ones_like(norm))
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(STEPS):
        g = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * g + c * torch.matmul(g, g), x)
    return x.transpose(1, 2) if tall else x


def _muon_plain(s):
    s["M"].mul_(MOMENTUM).add_(s["G"])
    o = _ortho_plain(s["G"] + MOMENTUM * s["M"])
    s["W"].mul_(1.0 - s["lr"] * DECAY).sub_(s["lr"] * _scale(s) * o)
    return dict(W=s["W"], M=s["M"])


# ------------------------------------------------------------------ one pass
def run(s):
    if not own:
        if s["op"].startswith("linear"):
            return _linear_plain(s)
        return _muon_plain(s) if s["op"] == "muon" else dict(O=_ortho_plain(s["G"]).to(BF))
    plan = s["plan"]
    if s["op"] == "ortho":
        return dict(O=plan.orthogonalize(s["G"]))
    if s["op"] == "muon":
        plan.step(s["W"], s["M"], s["G"], s["lr"])
        return dict(W=s["W"], M=s["M"])
    out = {}
    if s["op"] == "linear_step":
        plan.load(s["W"])
    if s["op"] != "linear_bwd":
        out["Y"] = plan.forward(s["X"])
    if s["op"] != "linear_fwd":
        out["dX"], out["dW"] = plan.backward(s["dY"], dW=s.get("dW"), accumulate=s["accumulate"])
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"].startswith("linear"):
        T, K, N = case["tokens"], case["inputs"], case["outputs"]
        fwd, bwd = case["op"] != "linear_bwd", case["op"] != "linear_fwd"
        codes = lambda n: n * (1.0 + 1.0 / BLOCK)  # noqa: E731
        bytes_ = N * K * (1.0 + 1.0 / BLOCK ** 2) if case["op"] != "linear_step" else 2.0 * N * K
        if fwd:
            bytes_ += 2.0 * T * K + 2.0 * T * N
        if bwd:
            bytes_ += 2.0 * T * N + 2.0 * T * K + (8.0 if case["accumulate"] else 4.0) * N * K
            bytes_ += codes(T * K) if not fwd else 0.0
        return dict(bytes=bytes_, flops=2.0 * T * K * N * (fwd + 2 * bwd))
    n, r, c = case["batch"], case["rows"], case["cols"]
    small, elems = min(r, c), n * r * c
    # of the two symmetric products one half
    flops = STEPS * n * (3.0 * small * r * c + small ** 3)
    return dict(bytes=elems * (20.0 if case["op"] == "muon" else (4.0 if case["half"] else 6.0)),
                flops=flops)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _e4m3_exact(v):
    """The nearest number of three mantissa bits (ties to even), steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step


def _rounded_exact(x, rows):
    """x [R][C] in 64 bits, each block of `rows` x 128 rounded in the steps of its own scale."""
    out = x.double().clone()
    R, C = x.shape
    for c0 in range(0, C, BLOCK):
        part = out[:, c0:c0 + BLOCK]
        top = part.abs().amax(1)
        if rows > 1:
            top = torch.cat([t.max().expand(t.numel()) for t in top.split(rows)])
        k = torch.floor(torch.log2(448.0 / top.clamp(min=1e-300)))
        # log2 may be off at a border: settle it by the inequality itself
        k = torch.where(top * torch.exp2(k) > 448.0, k - 1, k)
        k = torch.where(top * torch.exp2(k + 1) <= 448.0, k + 1, k).clamp(max=126)
        unit = torch.exp2(torch.where(top > 0, k, torch.zeros_like(k)))[:, None]
        part.copy_(_e4m3_exact(part * unit) / unit)
    return out


def _linear_exact(s):
    out = {}
    if s["op"] == "linear_step":
        w = _rounded_exact(s["W"], BLOCK)
    else:
        w = s["Wq"].double()
        for i in range(s["We"].shape[0]):
            for j in range(s["We"].shape[1]):
                w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= \
                    2.0 ** int(s["We"][i, j])
    if s["op"] != "linear_bwd":
        out["Y"] = torch.einsum("tk,nk->tn", _rounded_exact(s["X"], 1), w)
    if s["op"] != "linear_fwd":
        out["dX"] = torch.einsum("tn,nk->tk", _rounded_exact(s["dY"], 1), w)
        x = _rounded_exact(s["X"].t(), 1)
        out["dW"] = torch.einsum("nt,kt->nk", _rounded_exact(s["dY"].t(), 1), x)
        if s["accumulate"]:
            out["dW"] = out["dW"] + s["dW"].double()
    return out


def _ortho_exact(u):
    a, b, c = COEF
    out = torch.empty(u.shape, dtype=F64, device=DEV)
    for i in range(u.shape[0]):
        x = u[i].double()
        size = torch.linalg.matrix_norm(x)
        x = x / size if size > 0 else x
        for _ in range(STEPS):
            if x.shape[0] <= x.shape[1]:
                g = x @ x.mT
                y = g @ x
                x = a * x + b * y + c * (g @ y)
            else:
                g = x.mT @ x
                y = x @ g
                x = a * x + b * y + c * (y @ g)
        out[i] = x
    return out


def exact(case, seed):
    small = min(case.get("rows", 0), case.get("cols", 0))
    if case["op"] in ("ortho", "muon") and \
            case["batch"] * case["rows"] * case["cols"] * small > 3e11:
        return None  # about 6 STEPS times as many operations in 64 bits
    s = prepare(case, seed)
    if case["op"].startswith("linear"):
        return _linear_exact(s)
    G = s["G"].double()
    if case["op"] == "ortho":
        return dict(O=_ortho_exact(G))
    M = MOMENTUM * s["M"].double() + G
    O = _ortho_exact(G + MOMENTUM * M)
    lr = s["lr"].double()
    return dict(W=(1.0 - lr * DECAY) * s["W"].double() - lr * _scale(s) * O, M=M)
