"""Cases and plain forms of the operators at the two ends of a language model that
shares one table W [V, H] between its embedding and its head: the log probabilities of
given tokens (with entropy and top alternatives), the root-mean-square norm with the
residual's addition in front of the head, and the embedding lookup with its gradient.

With ``own`` false, ``run`` computes an operator from elementary torch operations in 32
bits; with ``own`` true it calls the framework.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100
EPS = 1e-6


def _lp(name, train, dtype, N, H, V, top_k, softcap, temperature, ignored, law):
    return dict(name=name, op="logprobs", train=train, dtype=dtype, N=N, H=H, V=V, top_k=top_k,
                softcap=softcap, temperature=temperature, ignored=ignored, law=law)


def _norm(name, train, dtype, N, H, residual, offset):
    return dict(name=name, op="rms_norm", train=train, dtype=dtype, N=N, H=H, residual=residual,
                offset=offset)


def _emb(name, train, dtype, N, H, V, law, padded):
    return dict(name=name, op="embedding", train=train, dtype=dtype, N=N, H=H, V=V, law=law,
                padded=padded)


def listed():
    return [
        # one sequence decoding: its next token's log probability and 8 alternatives
        _lp("logprobs-decode-1", False, "bf16", 1, 4096, 131072, 8, 0.0, 1.0, 0.0, "zipf"),
        # a serving batch of 48 sequences, capped logits, sampling temperature, 20 alternatives
        _lp("logprobs-decode-48", False, "bf16", 48, 3584, 256000, 20, 30.0, 0.7, 0.0, "uniform"),
        # prompts scored on a small head, 5 alternatives for each position
        _lp("logprobs-score-small", False, "bf16", 2048, 1024, 32000, 5, 0.0, 1.0, 0.05, "uniform"),
        # long prompts scored on a large head, the prompts' first quarter left out
        _lp("logprobs-score-large", False, "bf16", 8192, 4096, 131072, 8, 0.0, 1.0, 0.25, "zipf"),
        # a policy-gradient step with an entropy term, small head
        _lp("logprobs-train-small", True, "bf16", 2048, 1024, 32000, 0, 0.0, 1.0, 0.05, "uniform"),
        # the same in float32 at odd sizes, with capped logits and a temperature
        _lp("logprobs-train-odd-f32", True, "f32", 257, 515, 5003, 3, 30.0, 1.3, 0.1, "uniform"),
        # the same on a large head
        _lp("logprobs-train-large", True, "bf16", 4096, 4096, 131072, 0, 0.0, 1.0, 0.1, "zipf"),
        # the final norm of one decoding step of 16 sequences
        _norm("norm-decode-16", False, "bf16", 16, 4096, True, 0.0),
        # the final norm of a training batch, forward and backward
        _norm("norm-train", True, "bf16", 8192, 4096, True, 0.0),
        # odd width, float32, no residual, weights stored as their distance from one
        _norm("norm-train-odd-f32", True, "f32", 1000, 1029, False, 1.0),
        # prompts looked up in the small table
        _emb("embed-lookup", False, "bf16", 2048, 1024, 32000, "uniform", 0.05),
        # a training batch: lookup and the whole table's gradient, frequent tokens repeated
        _emb("embed-train", True, "bf16", 16384, 4096, 131072, "zipf", 0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "rms_norm", "embedding"])
    train = rng.random() < 0.5
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    law = rng.choice(["zipf", "uniform"])
    if op == "logprobs":
        # float32 heads are small ones; a training draw keeps below the listed step's work
        most = (512, 1024, 32000) if dtype == "f32" else (4096 if train else 8192, 4096, 131072)
        case = _lp("", train, dtype, _log_int(rng, 1, most[0]), _log_int(rng, 64, most[1]),
                   _log_int(rng, 300, most[2]), rng.choice([0, 1, 4, 10, 20]),
                   rng.choice([0.0, 30.0]), rng.choice([1.0, 0.7, 1.3]),
                   rng.choice([0.0, 0.1, 0.25]), law)
    elif op == "rms_norm":
        case = _norm("", train, dtype, _log_int(rng, 1, 8192),
                     _log_int(rng, 64, 2048 if dtype == "f32" else 4096), rng.random() < 0.7,
                     rng.choice([0.0, 1.0]))
    else:
        case = _emb("", train, dtype, _log_int(rng, 1, 16384),
                    _log_int(rng, 64, 2048 if dtype == "f32" else 4096),
                    _log_int(rng, 300, 131072), law, rng.choice([0.0, 0.1]))
    del case["name"]
    return case


# ---- inputs -----------------------------------------------------------------------------

def _tokens(case, g):
    """Token ids: uniform, or frequent ids far more often than rare ones (Zipf 1.1)."""
    N, V = case["N"], case["V"]
    if case["law"] == "uniform":
        return torch.randint(0, V, (N,), generator=g, device="cuda")
    w = torch.arange(1, V + 1, dtype=torch.float64, device="cuda").pow(-1.1)
    cdf = torch.cumsum(w, 0) / w.sum()
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    return torch.searchsorted(cdf, u).clamp_(0, V - 1)


def _grid(x, step):
    """x rounded to whole steps, at most 255 of them: exact in bf16. Products of such
    values and their sums over a row stay below 2^24 steps, so every float32 sum of
    them is exact in any order, and which alternative ranks higher, ties included, does
    not depend on how a logit was summed."""
    return (x / step).round_().clamp_(-255, 255) * step


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    N, H, dt = case["N"], case["H"], DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "rms_norm":
        s = dict(case=case, x=(2.0 * randn(N, H)).to(dt), residual=None,
                 weight=(1.0 - case["offset"] + 0.1 * randn(H)).to(dt))
        if case["residual"]:
            s["residual"] = (4.0 * randn(N, H)).to(dt)
        if case["train"]:
            s["dy"] = (0.01 * randn(N, H)).to(dt)
            s["ds"] = (0.01 * randn(N, H)).to(dt) if case["residual"] else None
        return s
    V, tokens = case["V"], _tokens(case, g)
    if case["op"] == "embedding":
        pad = torch.rand(N, generator=g, device="cuda") < case["padded"]
        s = dict(case=case, tokens=torch.where(pad, V - 1, tokens), W=(0.02 * randn(V, H)).to(dt))
        if case["train"]:
            s["dout"] = (0.01 * randn(N, H)).to(dt)
        return s
    # logits with a spread of about 1.3, and the given token's raised by up to 14, as a
    # trained model's are: some tokens nearly certain, others lost in the tail
    std = 1.28 / math.sqrt(H)
    W = _grid(std * randn(V, H), 2.0 ** math.floor(math.log2(std / 32)))
    gain = 14.0 * torch.rand(N, 1, generator=g, device="cuda")
    h = _grid(randn(N, H) + gain / (H * std * std) * W[tokens], 2.0 ** -5)
    n_ign = int(case["ignored"] * N)
    tokens[torch.randperm(N, generator=g, device="cuda")[:n_ign]] = IGNORE
    s = dict(case=case, h=h.to(dt), W=W.to(dt), tokens=tokens)
    if case["train"]:
        s["grad_logp"] = randn(N) / N
        s["grad_entropy"] = (-0.02 / N) * torch.rand(N, generator=g, device="cuda")
    return s


# ---- the plain forms --------------------------------------------------------------------

def _ranked(z, k):
    """The k largest logits of each row, equal ones by lowest index: a 64-bit key of the
    logit's order and the index makes every entry distinct."""
    V = z.shape[1]
    bits = (z + 0.0).view(torch.int32)
    order = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    key = (order.to(torch.int64) << 32) + (V - 1 - torch.arange(V, device=z.device))
    return V - 1 - (torch.topk(key, min(k, V), dim=1).values & 0xFFFFFFFF)


def _plain_logprobs(s):
    c, tokens = s["case"], s["tokens"]
    h, W = s["h"].float(), s["W"].float()
    live = tokens != IGNORE
    z = h @ W.t()
    cap, T = c["softcap"], c["temperature"]
    x = (cap * torch.tanh(z / cap) if cap else z) / T
    top = x.max(dim=1, keepdim=True).values
    e = torch.exp(x - top)
    total = e.sum(dim=1, keepdim=True)
    log_total = torch.log(total)
    at = tokens.clamp_min(0).unsqueeze(1)
    zero = torch.zeros((), device=z.device)
    p = e / total
    entropy = log_total[:, 0] - (p * (x - top)).sum(dim=1)
    out = dict(logp=torch.where(live, ((x.gather(1, at) - top) - log_total)[:, 0], zero),
               entropy=torch.where(live, entropy, zero),
               lse=torch.where(live, (top + log_total)[:, 0], zero))
    if c["top_k"]:
        ids = _ranked(z, c["top_k"])
        out["top_logp"] = torch.where(live[:, None], (x.gather(1, ids) - top) - log_total,
                                      -math.inf)
        out["top_ids"] = torch.where(live[:, None], ids, -1)
    if c["train"]:
        a = torch.where(live, s["grad_logp"], zero)[:, None]
        b = torch.where(live, s["grad_entropy"], zero)[:, None]
        G = -p * (a + b * ((x - top) - log_total + entropy[:, None]))
        G.scatter_add_(1, at, a)
        G = G / T
        if cap:
            t = torch.tanh(z / cap)
            G = G * (1 - t * t)
        out["dH"] = (G @ W).to(s["h"].dtype)
        out["dW"] = (G.t() @ h).to(s["W"].dtype)
    return out


def _plain_rms_norm(s):
    c, dt = s["case"], s["x"].dtype
    x = s["x"].float()
    r = (x + s["residual"].float()).to(dt) if c["residual"] else s["x"]
    v = r.float()
    w = s["weight"].float() + c["offset"]
    rstd = torch.rsqrt((v * v).mean(dim=1) + EPS)
    n = v * rstd[:, None]
    out = dict(y=(n * w).to(dt), rstd=rstd)
    if c["residual"]:
        out["s"] = r
    if c["train"]:
        dy = s["dy"].float()
        g = dy * w
        dx = rstd[:, None] * (g - n * (g * n).mean(dim=1, keepdim=True))
        if s["ds"] is not None:
            dx = dx + s["ds"].float()
        out["dx"] = dx.to(dt)
        out["dw"] = (dy * n).sum(dim=0).to(dt)
    return out


def _plain_embedding(s):
    c, tokens, W = s["case"], s["tokens"], s["W"]
    scale = math.sqrt(c["H"])
    live = (tokens != c["V"] - 1)[:, None]
    out = dict(out=(W[tokens].float() * scale * live).to(W.dtype))
    if c["train"]:
        dW = torch.zeros(c["V"], c["H"], device=W.device)
        dW.index_add_(0, tokens, s["dout"].float() * live)
        out["dW"] = (dW * scale).to(W.dtype)
    return out


# ---- the framework's calls ----------------------------------------------------------------

def _own_logprobs(s):
    import lm_head_linear_amd as flce
    c = s["case"]
    kw = dict(ignore_index=IGNORE, softcap=c["softcap"], temperature=c["temperature"])
    r = flce.flce_logprobs(s["h"], s["W"], s["tokens"], top_k=c["top_k"], **kw)
    out = dict(logp=r.logp, entropy=r.entropy, lse=r.lse)
    if c["top_k"]:
        out["top_logp"], out["top_ids"] = r.top_logp, r.top_ids
    if c["train"]:
        out["dH"], out["dW"] = flce.flce_logprobs_backward(
            s["h"], s["W"], s["tokens"], r.lse, r.entropy, s["grad_logp"], s["grad_entropy"], **kw)
    return out


def _own_rms_norm(s):
    import lm_head_linear_amd as flce
    c = s["case"]
    y, r, rstd = flce.flce_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS,
                                    weight_offset=c["offset"])
    out = dict(y=y, rstd=rstd)
    if c["residual"]:
        out["s"] = r
    if c["train"]:
        out["dx"], out["dw"] = flce.flce_rms_norm_backward(
            s["dy"], r, s["weight"], rstd, s["ds"], weight_offset=c["offset"])
    return out


def _own_embedding(s):
    import lm_head_linear_amd as flce
    c = s["case"]
    kw = dict(scale=math.sqrt(c["H"]), padding_index=c["V"] - 1)
    out = dict(out=flce.flce_embedding(s["tokens"], s["W"], **kw))
    if c["train"]:
        out["dW"] = flce.flce_embedding_backward(s["tokens"], s["dout"], c["V"], **kw)
    return out


PLAIN = {"logprobs": _plain_logprobs, "rms_norm": _plain_rms_norm, "embedding": _plain_embedding}
OWN = {"logprobs": _own_logprobs, "rms_norm": _own_rms_norm, "embedding": _own_embedding}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


def work(case):
    N, H, e = case["N"], case["H"], DTYPES[case["dtype"]].itemsize
    if case["op"] == "rms_norm":
        res = case["residual"]
        b = N * H * e * (4 if res else 2) + H * e + 4 * N
        if case["train"]:
            b += N * H * e * (3 if res else 2) + H * e
        return {"bytes": b, "flops": N * H * (12 if case["train"] else 4)}
    V = case["V"]
    if case["op"] == "embedding":
        b = N * 8 + 2 * min(N, V) * H * e + (N - min(N, V)) * H * e
        if case["train"]:
            b += N * H * e + V * H * e
        return {"bytes": b, "flops": N * H * (2 if case["train"] else 1)}
    live = N - int(case["ignored"] * N)
    b = (N + V) * H * e + N * 8 + 12 * N + 12 * N * case["top_k"]
    f = 2.0 * live * H * V
    if case["train"]:
        b += (N + V) * H * e + 8 * N
        f *= 3
    return {"bytes": b, "flops": f}


# ---- the definitions in 64 bits -------------------------------------------------------------

def _exact_logprobs(s):
    c = s["case"]
    W = s["W"].double()
    V, K, cap, T = c["V"], min(c["top_k"], c["V"]), c["softcap"], c["temperature"]
    rows = max(1, (1 << 27) // V)
    cols = {n: [] for n in ("logp", "entropy", "lse", "top_logp", "top_ids", "dH")}
    dW = torch.zeros_like(W) if c["train"] else None
    for r0 in range(0, c["N"], rows):
        h = s["h"][r0:r0 + rows].double()
        tok = s["tokens"][r0:r0 + rows]
        live = tok != IGNORE
        z = torch.matmul(h, W.T)
        x = (cap * torch.tanh(z / cap) if cap > 0 else z) / T
        lse = torch.logsumexp(x, 1)
        lp = x - lse[:, None]
        p = lp.exp()
        at = torch.where(live, tok, 0)[:, None]
        ent = -(p * lp).sum(1)
        cols["logp"].append(lp.gather(1, at)[:, 0] * live)
        cols["entropy"].append(ent * live)
        cols["lse"].append(lse * live)
        if K:
            order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :K]
            cols["top_ids"].append(torch.where(live[:, None], order, -1))
            cols["top_logp"].append(lp.gather(1, order).masked_fill(~live[:, None], -math.inf))
        if c["train"]:
            a = s["grad_logp"][r0:r0 + rows].double()[:, None]
            b = s["grad_entropy"][r0:r0 + rows].double()[:, None]
            hot = torch.zeros_like(p).scatter_(1, at, 1.0)
            gx = a * (hot - p) - b * p * (lp + ent[:, None])
            if cap > 0:
                gx = gx * (1 - torch.tanh(z / cap) ** 2)
            gz = gx * live[:, None] / T
            cols["dH"].append(gz @ W)
            dW.addmm_(gz.T, h)
    out = {n: torch.cat(v) for n, v in cols.items() if v}
    if c["train"]:
        out["dW"] = dW
    return out


def _exact_rms_norm(s):
    c = s["case"]
    v = s["x"].double()
    if c["residual"]:
        v = (v + s["residual"].double()).to(s["x"].dtype).double()   # the stored sum is rounded
    w = s["weight"].double() + c["offset"]
    std = ((v ** 2).sum(1) / c["H"] + EPS).sqrt()
    out = dict(y=v / std[:, None] * w, rstd=1 / std)
    if c["residual"]:
        out["s"] = v
    if c["train"]:
        dy = s["dy"].double()
        proj = (dy * w * v).sum(1) / (c["H"] * std ** 3)
        out["dx"] = dy * w / std[:, None] - proj[:, None] * v
        if s["ds"] is not None:
            out["dx"] = out["dx"] + s["ds"].double()
        out["dw"] = (dy * v / std[:, None]).sum(0)
    return out


def _exact_embedding(s):
    c, tokens = s["case"], s["tokens"]
    scale = math.sqrt(c["H"])
    keep = (tokens != c["V"] - 1).double()[:, None]
    out = dict(out=s["W"].double()[tokens] * keep * scale)
    if c["train"]:
        dW = torch.zeros(c["V"], c["H"], dtype=torch.float64, device="cuda")
        out["dW"] = dW.index_add(0, tokens, s["dout"].double() * keep) * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "rms_norm": _exact_rms_norm,
            "embedding": _exact_embedding}[case["op"]](s)
