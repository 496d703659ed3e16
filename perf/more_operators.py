"""Cases and plain forms of operators that stand before and after a language model's
head: the linear transform in front of it (a matrix product with bias, activation and
residual in its epilogue), dropout from a counter-based generator (alone, with the
residual's addition, and with the addition and the norm), and the sampling of the next
token from the head's logits with temperature, top-k, top-p and min-p.

With ``own`` false, ``run`` computes an operator from elementary torch operations in 32
bits (sampling's weights and sums, whose borders decide a token, in 64); with ``own``
true it calls the framework.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _sample(name, head, dtype, N, H, V, temperature, top_k, top_p, min_p, softcap, masked, per_row):
    return dict(name=name, op="sample", head=head, dtype=dtype, N=N, H=H, V=V,
                temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, softcap=softcap,
                masked=masked, per_row=per_row)


def _linear(name, train, dtype, N, I, O, activation, bias, residual):
    return dict(name=name, op="linear", train=train, dtype=dtype, N=N, I=I, O=O,
                activation=activation, bias=bias, residual=residual)


def _dropout(name, train, dtype, N, H, p, residual, norm):
    return dict(name=name, op="dropout", train=train, dtype=dtype, N=N, H=H, p=p,
                residual=residual, norm=norm)


def listed():
    return [
        # one sequence decoding: its next token from logits at hand
        _sample("sample-logits-1", False, "f32", 1, 0, 131072, 0.7, 50, 0.9, 0.0, 0.0, 0.0, False),
        # a serving batch whose requests each bring their own settings, bf16 logits, ids that a
        # grammar forbids
        _sample("sample-requests-128", False, "bf16", 128, 0, 32000, 0.8, 40, 0.95, 0.05, 0.0, 0.3, True),
        # many rollouts at once, no limit on the count of candidates
        _sample("sample-rollouts-256", False, "f32", 256, 0, 131072, 1.0, 0, 0.95, 0.0, 0.0, 0.0, False),
        # a serving batch of 48 sequences through a capped head
        _sample("sample-head-48", True, "bf16", 48, 3584, 256000, 0.7, 20, 0.95, 0.0, 30.0, 0.0, False),
        # the transform in front of the head, one decoding step of 16 sequences
        _linear("linear-decode-16", False, "bf16", 16, 4096, 4096, "silu", True, True),
        # a small head's transform, forward and backward
        _linear("linear-train-small", True, "bf16", 2048, 1024, 1024, "gelu", True, True),
        # odd sizes in float32, no residual
        _linear("linear-train-odd-f32", True, "f32", 257, 515, 701, "gelu_tanh", True, False),
        # a large head's transform, forward and backward
        _linear("linear-train-large", True, "bf16", 8192, 4096, 4096, "silu", True, True),
        # embeddings of a small model's batch, forward and backward
        _dropout("dropout-embeddings", True, "bf16", 2048, 1024, 0.1, False, False),
        # odd width, float32, added to the residual
        _dropout("dropout-residual-odd-f32", True, "f32", 1000, 1029, 0.5, True, False),
        # a training batch: dropped out, added to the residual
        _dropout("dropout-residual-large", True, "bf16", 8192, 4096, 0.1, True, False),
        # the same and the norm of the sum, in front of the head
        _dropout("dropout-norm-large", True, "bf16", 8192, 4096, 0.1, True, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "linear", "linear", "dropout"])
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    train = rng.random() < 0.6
    if op == "sample":
        head = rng.random() < 0.3
        f32_head = head and dtype == "f32"
        case = _sample("", head, dtype, _log_int(rng, 1, 48 if head else 256),
                       _log_int(rng, 64, 1024 if f32_head else 3584) if head else 0,
                       _log_int(rng, 300, 32000 if f32_head else 131072),
                       rng.choice([0.0, 0.7, 1.0, 1.3]), rng.choice([0, 0, 1, 20, 50, 1000]),
                       rng.choice([1.0, 0.5, 0.9, 0.95]), rng.choice([0.0, 0.0, 0.05]),
                       rng.choice([0.0, 30.0]), 0.0 if head else rng.choice([0.0, 0.3, 0.9]),
                       rng.random() < 0.4)
    elif op == "linear":
        most = (1024, 1024) if dtype == "f32" else (8192, 4096)
        case = _linear("", train, dtype, _log_int(rng, 1, most[0]), _log_int(rng, 64, most[1]),
                       _log_int(rng, 64, most[1]),
                       rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                       rng.random() < 0.7, rng.random() < 0.6)
    else:
        norm = rng.random() < 0.4
        case = _dropout("", train, dtype, _log_int(rng, 1, 8192),
                        _log_int(rng, 64, 2048 if dtype == "f32" else 4096),
                        rng.choice([0.05, 0.1, 0.3, 0.5]), norm or rng.random() < 0.6, norm)
    del case["name"]
    return case


# ---- inputs -----------------------------------------------------------------------------

def _grid(x, step):
    """x rounded to whole steps, at most 255 of them: exact in bf16. Products of such
    values and their sums over a row stay below 2^24 steps, so every float32 sum of them is
    exact in any order, and the logits do not depend on how they were summed."""
    return (x / step).round_().clamp_(-255, 255) * step


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    N, dt = case["N"], DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case=case)
    if case["op"] == "linear":
        I, O = case["I"], case["O"]
        x, weight, bias = randn(N, I), randn(O, I) / math.sqrt(I), 0.1 * randn(O)
        if case["activation"] == "relu":
            # exact sums: which side of zero a value lies on does not depend on their order
            x, bias = _grid(x, 2.0 ** -5), _grid(bias, 2.0 ** -9)
            weight = _grid(weight, 2.0 ** (math.floor(-0.5 * math.log2(I)) - 5))
        s.update(x=x.to(dt), weight=weight.to(dt), bias=bias.to(dt) if case["bias"] else None,
                 residual=(2.0 * randn(N, O)).to(dt) if case["residual"] else None)
        if case["train"]:
            s["dy"] = (0.01 * randn(N, O)).to(dt)
        return s
    if case["op"] == "dropout":
        H = case["H"]
        s.update(x=randn(N, H).to(dt), residual=(4.0 * randn(N, H)).to(dt) if case["residual"] else None,
                 seed=int(torch.randint(0, 1 << 62, (1,), generator=g, device="cuda")),
                 offset=int(torch.randint(0, 1 << 40, (1,), generator=g, device="cuda")))
        if case["norm"]:
            s["weight"] = (1.0 + 0.1 * randn(H)).to(dt)
        if case["train"]:
            s["dout"] = (0.01 * randn(N, H)).to(dt)
            s["ds"] = (0.01 * randn(N, H)).to(dt) if case["norm"] else None
        return s
    V, H = case["V"], case["H"]
    s["uniforms"] = rand(N)
    # logits with a spread of about 2 and a few raised ones, as a trained model's have
    if case["head"]:
        std = 2.0 / math.sqrt(H)
        W = _grid(std * randn(V, H), 2.0 ** math.floor(math.log2(std / 32)))
        best = torch.randint(0, V, (N,), generator=g, device="cuda")
        h = _grid(randn(N, H) + 10.0 * rand(N, 1) / (H * std * std) * W[best], 2.0 ** -5)
        s.update(h=h.to(dt), W=W.to(dt))
    else:
        z = 2.0 * randn(N, V)
        up = torch.randint(0, V, (N, 8), generator=g, device="cuda")
        z.scatter_add_(1, up, 12.0 * rand(N, 8))
        if case["masked"]:
            z.masked_fill_(rand(N, V) < case["masked"], -math.inf)
        s["logits"] = z.to(dt)
    for name in ("temperature", "top_k", "top_p", "min_p"):
        s[name] = case[name]
    if case["per_row"]:
        # each request its own: a quarter greedy, the others around the case's settings
        greedy = rand(N) < 0.25
        s["temperature"] = torch.where(greedy, 0.0, (case["temperature"] or 1.0) * (0.5 + rand(N)))
        s["top_k"] = torch.randint(0, 2 * case["top_k"] + 1, (N,), generator=g, device="cuda",
                                   dtype=torch.int32)
        s["top_p"] = (case["top_p"] + 0.2 * (rand(N) - 0.5)).clamp_(max=1.0)
        s["min_p"] = case["min_p"] * 2 * rand(N)
    return s


# ---- the plain forms --------------------------------------------------------------------

def _column(v, N, dtype):
    if isinstance(v, torch.Tensor):
        return v.to(dtype)[:, None]
    # a scalar setting travels as float32
    return torch.full((N, 1), v, dtype=torch.float32, device="cuda").to(dtype)


def _plain_sample(s):
    c = s["case"]
    N, V, cap = c["N"], c["V"], c["softcap"]
    z = s["h"].float() @ s["W"].float().t() if c["head"] else s["logits"].float()
    T, top_p, min_p = (_column(s[n], N, torch.float64) for n in ("temperature", "top_p", "min_p"))
    top_k = _column(s["top_k"], N, torch.int64)
    # greedy is a top-1 of any temperature
    top_k = torch.where((top_k <= 0) | (top_k > V), V, top_k)
    top_k = torch.where(T == 0, 1, top_k)
    T = torch.where(T == 0, 1.0, T)
    # ranks: largest first, equal ones by lowest index (a 64-bit key of both)
    bits = (z + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64)
    key = (order << 32) + (V - 1 - torch.arange(V, device=z.device))
    rank = torch.argsort(key, dim=1, descending=True)
    x = z.double()
    if cap:
        x = cap * torch.tanh(x / cap)
    w = torch.exp((x - x.max(dim=1, keepdim=True).values) / T)
    r = torch.gather(w, 1, rank)
    r = r * (torch.arange(V, device=z.device) < top_k)
    above = torch.cumsum(r, 1) - r
    keep = (r > 0) & (above < top_p * r.sum(1, keepdim=True)) & (r >= min_p)
    keep[:, 0] = True
    w = w * torch.zeros_like(keep).scatter_(1, rank, keep)
    cum = torch.cumsum(w, 1)
    total = w.sum(1, keepdim=True)
    token = (cum <= s["uniforms"].double()[:, None] * total).sum(1, keepdim=True)
    # never behind the last kept one
    last = torch.where(w > 0, torch.arange(V, device=z.device), -1).max(1, keepdim=True).values
    token = torch.minimum(token, last)
    logp = torch.log(torch.gather(w, 1, token) / total)
    return dict(tokens=token[:, 0], logp=logp[:, 0].float())


def _act(kind, z):
    if kind == "relu":
        return torch.where(z > 0, z, 0.0)
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(kind, z):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if kind == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    return torch.ones_like(z)


def _plain_linear(s):
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    z = x @ w.t()
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(c["activation"], z)
    if c["residual"]:
        y = y + s["residual"].float()
    out = dict(y=y.to(dt))
    if c["train"]:
        dz = s["dy"].float() * _act_slope(c["activation"], z)
        out["dx"] = (dz @ w).to(dt)
        out["dweight"] = (dz.t() @ x).to(dt)
        if c["bias"]:
            out["dbias"] = dz.sum(0).to(dt)
    return out


M32 = 0xFFFFFFFF


def _words(s):
    """Ten rounds of Philox 4x32 (Salmon et al., SC 2011) of the counter (column / 8, row,
    offset) under the key (seed): eight 16-bit numbers for eight columns."""
    N, H = s["case"]["N"], s["case"]["H"]
    c = [torch.arange((H + 7) // 8, device="cuda")[None, :].expand(N, -1),
         torch.arange(N, device="cuda")[:, None].expand(-1, (H + 7) // 8)]
    c += [torch.full_like(c[0], s["offset"] & M32), torch.full_like(c[0], s["offset"] >> 32)]
    k0, k1 = s["seed"] & M32, s["seed"] >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & M32) ^ c[1] ^ k0, b & M32, ((a >> 32) & M32) ^ c[3] ^ k1, a & M32]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    halves = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], dim=2)
    return halves.reshape(N, -1)[:, :H]


def _plain_dropout(s):
    c, dt = s["case"], s["x"].dtype
    t = min(int(c["p"] * 65536 + 0.5), 65535)
    keep, scale = _words(s) >= t, 65536 / (65536 - t)
    x = torch.where(keep, s["x"].float() * scale, 0.0)
    if c["residual"]:
        x = x + s["residual"].float()
    r = x.to(dt)
    if not c["norm"]:
        out = dict(out=r)
        if c["train"]:
            out["dx"] = torch.where(keep, s["dout"].float() * scale, 0.0).to(dt)
        return out
    v, w = r.float(), s["weight"].float()
    rstd = torch.rsqrt((v * v).mean(dim=1) + EPS)
    n = v * rstd[:, None]
    out = dict(y=(n * w).to(dt), s=r, rstd=rstd)
    if c["train"]:
        dy = s["dout"].float()
        g = dy * w
        d = rstd[:, None] * (g - n * (g * n).mean(dim=1, keepdim=True)) + s["ds"].float()
        out["dresidual"] = d.to(dt)
        out["dx"] = torch.where(keep, d * scale, 0.0).to(dt)
        out["dweight"] = (dy * n).sum(dim=0).to(dt)
    return out


# ---- the framework's calls ----------------------------------------------------------------

def _own_sample(s):
    import lm_head_linear_amd as flce
    kw = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
              softcap=s["case"]["softcap"])
    if s["case"]["head"]:
        r = flce.flce_sample(s["h"], s["W"], s["uniforms"], **kw)
    else:
        r = flce.flce_sample_logits(s["logits"], s["uniforms"], **kw)
    return dict(tokens=r.tokens, logp=r.logp)


def _own_linear(s):
    import lm_head_linear_amd as flce
    c = s["case"]
    y, slope = flce.flce_linear(s["x"], s["weight"], s["bias"], s["residual"],
                            activation=c["activation"], save_slope=c["train"])
    out = dict(y=y)
    if c["train"]:
        out["dx"], out["dweight"], db = flce.flce_linear_backward(
            s["dy"], s["x"], s["weight"], slope, bias=c["bias"])
        if c["bias"]:
            out["dbias"] = db
    return out


def _own_dropout(s):
    import lm_head_linear_amd as flce
    c = s["case"]
    kw = dict(p=c["p"], seed=s["seed"], offset=s["offset"])
    if not c["norm"]:
        out = dict(out=flce.flce_dropout(s["x"], s["residual"], **kw))
        if c["train"]:
            out["dx"] = flce.flce_dropout_backward(s["dout"], **kw)
        return out
    y, r, rstd = flce.flce_dropout_norm(s["x"], s["weight"], s["residual"], eps=EPS, **kw)
    out = dict(y=y, s=r, rstd=rstd)
    if c["train"]:
        out["dx"], out["dresidual"], out["dweight"] = flce.flce_dropout_norm_backward(
            s["dout"], r, s["weight"], rstd, s["ds"], **kw)
    return out


PLAIN = {"sample": _plain_sample, "linear": _plain_linear, "dropout": _plain_dropout}
OWN = {"sample": _own_sample, "linear": _own_linear, "dropout": _own_dropout}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


def work(case):
    N, e = case["N"], DTYPES[case["dtype"]].itemsize
    if case["op"] == "sample":
        H, V = case["H"], case["V"]
        settings = 16 * N if case["per_row"] else 0
        if case["head"]:
            return {"bytes": (N + V) * H * e + 16 * N + settings, "flops": 2.0 * N * H * V}
        return {"bytes": N * V * e + 16 * N + settings, "flops": 4 * N * V}
    if case["op"] == "linear":
        I, O = case["I"], case["O"]
        b = (N * I + O * I + N * O * (2 if case["residual"] else 1) + (O if case["bias"] else 0)) * e
        f = 2.0 * N * I * O
        if case["train"]:
            # dy in; dx, dweight, dbias out
            b += (N * O + N * I + O * I + (O if case["bias"] else 0)) * e
            f *= 3
        return {"bytes": b, "flops": f}
    H = case["H"]
    rows = 3 if case["residual"] else 2
    if case["norm"]:
        rows += 1
    if case["train"]:
        # dout to dx; with the norm dy, ds to dx, dresidual
        rows += 4 if case["norm"] else 2
    b = N * H * e * rows + (2 * H * e + 4 * N if case["norm"] else 0)
    return {"bytes": b, "flops": N * H * (16 if case["norm"] else 4)}


# ---- the definitions in 64 bits -------------------------------------------------------------

def _exact_sample(s):
    c = s["case"]
    tokens, logp = [], []

    def setting(name, i):
        v = s[name]
        if isinstance(v, torch.Tensor):
            return float(v[i])
        return float(torch.tensor(v, dtype=torch.float32))

    for i in range(c["N"]):
        if c["head"]:
            z = torch.mv(s["W"].double(), s["h"][i].double()) if c["N"] == 1 else s["_z"][i]
        else:
            z = s["logits"][i].double()
        ranked, at = torch.sort(z, descending=True, stable=True)
        T, k = setting("temperature", i), int(setting("top_k", i))
        if T == 0:
            T, k = 1.0, 1
        if not 0 < k < c["V"]:
            k = c["V"]
        ranked, at = ranked[:k], at[:k]
        if c["softcap"]:
            ranked = c["softcap"] * torch.tanh(ranked / c["softcap"])
        p = torch.softmax(ranked / T, 0)
        before = torch.cat([torch.zeros_like(p[:1]), torch.cumsum(p, 0)[:-1]])
        ok = (before < setting("top_p", i)) & (p >= setting("min_p", i) * p[0]) & (p > 0)
        ok[0] = True
        at, p = at[ok], p[ok]
        at, by_index = torch.sort(at)
        p = p[by_index] / p.sum()
        j = int(torch.searchsorted(torch.cumsum(p, 0), s["uniforms"][i].double(), right=True))
        j = min(j, p.numel() - 1)
        tokens.append(at[j])
        logp.append(torch.log(p[j]))
    return dict(tokens=torch.stack(tokens), logp=torch.stack(logp))


def _exact_linear(s):
    c = s["case"]
    w, x = s["weight"].double(), s["x"].double()
    z = torch.mm(x, w.T)
    if c["bias"]:
        z += s["bias"].double()
    z.requires_grad_(c["train"])
    a = {"none": lambda t: t * 1, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh"),
         "silu": torch.nn.functional.silu}[c["activation"]](z)
    out = dict(y=a.detach() + (s["residual"].double() if c["residual"] else 0.0))
    if c["train"]:
        dz, = torch.autograd.grad(a, z, s["dy"].double())
        out["dx"], out["dweight"] = torch.mm(dz, w), torch.mm(dz.T, x)
        if c["bias"]:
            out["dbias"] = dz.sum(0)
    return out


def _exact_keep(s, t):
    """The mask, a column of blocks at a time, products of 32 bits in halves of 16."""
    N, H = s["case"]["N"], s["case"]["H"]
    keep = torch.empty(N, (H + 7) // 8 * 8, dtype=torch.bool, device="cuda")

    def product(m, v):
        lo, hi = m * (v & 0xFFFF), m * (v >> 16)          # below 2^48 each
        low = lo + ((hi & 0xFFFF) << 16)
        return (hi >> 16) + (low >> 32), low & M32

    step = max(1, (1 << 21) // N)
    for b0 in range(0, (H + 7) // 8, step):
        cols = torch.arange(b0, min(b0 + step, (H + 7) // 8), device="cuda")
        x0 = cols.repeat(N, 1)
        x1 = torch.arange(N, device="cuda").unsqueeze(1).repeat(1, cols.numel())
        x2, x3 = torch.full_like(x0, s["offset"] % 2**32), torch.full_like(x0, s["offset"] // 2**32)
        for r in range(10):
            ka = (s["seed"] + r * 0x9E3779B9) % 2**32
            kb = (s["seed"] // 2**32 + r * 0xBB67AE85) % 2**32
            h0, l0 = product(0xD2511F53, x0)
            h2, l2 = product(0xCD9E8D57, x2)
            x0, x1, x2, x3 = h2 ^ x1 ^ ka, l2, h0 ^ x3 ^ kb, l0
        for i, v in enumerate((x0, x1, x2, x3)):
            keep[:, 8 * b0 + 2 * i:8 * int(cols[-1]) + 8:8] = v % 65536 >= t
            keep[:, 8 * b0 + 2 * i + 1:8 * int(cols[-1]) + 8:8] = v // 65536 >= t
    return keep[:, :H]


def _exact_dropout(s):
    c, dt = s["case"], s["x"].dtype
    t = min(math.floor(65536 * c["p"] + 0.5), 65535)
    factor = _exact_keep(s, t).double() * (65536 / (65536 - t))
    v = s["x"].double() * factor
    if c["residual"]:
        v = v + s["residual"].double()
    if not c["norm"]:
        out = dict(out=v)
        if c["train"]:
            out["dx"] = s["dout"].double() * factor
        return out
    stored = v.to(dt).double()                     # the norm is of the stored sum
    w = s["weight"].double()
    std = ((stored ** 2).sum(1) / c["H"] + EPS).sqrt()
    out = dict(y=stored / std[:, None] * w, s=v, rstd=1 / std)
    if c["train"]:
        dy = s["dout"].double()
        proj = (dy * w * stored).sum(1) / (c["H"] * std ** 3)
        out["dresidual"] = dy * w / std[:, None] - proj[:, None] * stored + s["ds"].double()
        out["dx"] = out["dresidual"] * factor
        out["dweight"] = (dy * stored / std[:, None]).sum(0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample" and case["head"] and case["N"] > 1:
        s["_z"] = torch.mm(s["h"].double(), s["W"].double().T)
    return {"sample": _exact_sample, "linear": _exact_linear,
            "dropout": _exact_dropout}[case["op"]](s)
