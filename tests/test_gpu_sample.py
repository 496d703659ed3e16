"""Sampling with temperature, top-k, top-p and min-p from given uniform numbers, against a
sorted float64 form on the CPU, with the weights' documented grain. Tokens have to be equal: the kernel decides to 2^-S of the
largest weight (2^-45 for 131072 logits), the float64 form to about 2^-50 of the mass, so that
the two part only where a border lies within some 1e-11 of the uniform number. logp is a
float64 logarithm rounded to float32: half a step, and 1e-9 for the weights' grain."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


def f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


def oracle(z, u, T=1.0, k=0, p=1.0, q=0.0, cap=0.0):
    """(token, logp) of one row, settings as float32 values."""
    z = z.double().cpu()
    V = z.numel()
    if bool(z.isnan().any()):
        return -1, math.nan
    if bool((z == -math.inf).all()):
        return -1, -math.inf
    order = torch.sort(z, descending=True, stable=True).indices
    if not T > 0:
        T, k = 1.0, 1
    k = V if k <= 0 or k > V else k
    top = z[order[0]]
    x = cap * torch.tanh(z / cap) if cap else z
    w = torch.exp((x - x[order[0]]) / T)
    w = torch.where(z == top, 1.0, torch.where(w.isnan() | (z == -math.inf), 0.0, w))
    grain = 2.0 ** min(51, 62 - math.ceil(math.log2(V)))   # weights are multiples of 1 / grain
    order = order[:k]
    r = torch.round(w[order] * grain) / grain
    above = torch.cumsum(r, 0) - r
    p = 0.0 if math.isnan(p) else p
    q = 0.0 if math.isnan(q) else min(max(q, 0.0), 1.0)
    ok = (w[order] >= q) & (r > 0)
    if p < 1:
        ok &= above < p * r.sum()
    ok[0] = True
    kept = torch.zeros(V, dtype=torch.float64)
    kept[order[ok]] = r[ok]
    cum = torch.cumsum(kept, 0)
    u = 0.0 if math.isnan(u) else min(max(u, 0.0), 1.0)
    at = int((cum <= u * cum[-1]).sum())
    at = min(at, int(kept.nonzero().max()))
    return at, float(torch.log(w[at] / cum[-1]))


def compare(r, z, u, **kw):
    for i in range(z.shape[0]):
        row = {n: (float(v[i]) if torch.is_tensor(v) else f32(v)) for n, v in kw.items()}
        row["k"] = int(row.get("k", 0))
        tok, lp = oracle(z[i], float(u[i]), **row)
        got, glp = int(r.tokens[i]), float(r.logp[i])
        assert got == tok, (i, got, tok, row, float(u[i]))
        same = glp == lp or (math.isnan(lp) and math.isnan(glp))
        assert same or abs(glp - lp) <= 2.0 ** -24 * abs(lp) * 1.01 + 1e-9, (i, glp, lp)


def run(z, u, T=1.0, k=0, p=1.0, q=0.0, cap=0.0):
    import lm_head_linear_amd as m
    return m.flce_sample_logits(z, u, temperature=T, top_k=k, top_p=p, min_p=q, softcap=cap)


def make(N, V, dt, seed, masked=0.0, step=0.0):
    g = torch.Generator().manual_seed(seed)
    z = 2.5 * torch.randn(N, V, generator=g)
    z[torch.arange(N), torch.randint(0, V, (N,), generator=g)] += 8 * torch.rand(N, generator=g)
    if step:
        z = (z / step).round() * step
    if masked:
        z[torch.rand(N, V, generator=g) < masked] = -math.inf
        z[:, 0] = 0
    return z.to(dt).cuda(), torch.rand(N, generator=g).cuda()


SETTINGS = [dict(), dict(T=0.7), dict(T=1.3, k=50), dict(k=1), dict(p=0.9), dict(T=0.5, p=0.3),
            dict(q=0.05), dict(T=0.8, k=40, p=0.95, q=0.02), dict(T=0.0), dict(k=1000, p=0.5),
            dict(cap=30.0, T=0.7, k=20, p=0.95), dict(cap=5.0), dict(T=1e-3), dict(T=50.0, p=0.99),
            dict(k=7), dict(T=2.0, q=1.0), dict(p=1e-6), dict(T=1e30, k=10)]
VOCABS = [(5, 1), (6, 2), (9, 7), (7, 63), (7, 64), (7, 65), (6, 130), (5, 1000), (5, 1029),
          (5, 2049), (4, 16384), (3, 16385), (3, 32000), (3, 50257), (2, 131072), (2, 200003)]


@pytest.mark.parametrize("N,V", VOCABS)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_vocabularies_and_settings(N, V, dt):
    for i, s in enumerate(SETTINGS):
        z, u = make(N, V, dt, i + V)
        compare(run(z, u, **s), z, u, **s)


@pytest.mark.parametrize("N", [1, 2, 17, 70, 300])
@pytest.mark.parametrize("V", [999, 8192])
def test_counts_of_rows(N, V):
    for i, s in enumerate((dict(T=0.9, p=0.9), dict(k=33), dict(T=1.0), dict(k=20, p=0.8, q=0.01))):
        z, u = make(N, V, torch.float32, i)
        compare(run(z, u, **s), z, u, **s)


@pytest.mark.parametrize("V", [65, 1000, 5000, 40000])
def test_ties_and_masks(V):
    """Logits on a coarse grid: most are equal to others; and most are masked."""
    for step, masked in ((0.5, 0.0), (4.0, 0.0), (1.0, 0.9), (0.0, 0.97), (100.0, 0.5)):
        for i, s in enumerate(SETTINGS):
            z, u = make(4, V, torch.float32, i, masked=masked, step=step)
            compare(run(z, u, **s), z, u, **s)
    z = torch.zeros(6, V, device="cuda")                  # all equal
    u = torch.tensor([0.0, 0.1, 0.5, 0.9, 0.999, 1.0], device="cuda")
    for s in SETTINGS:
        compare(run(z, u, **s), z, u, **s)


def test_rows_of_their_own_settings():
    g = torch.Generator().manual_seed(5)
    N = 60
    for V in (500, 33000):
        z, u = make(N, V, torch.float32, V)
        T = (torch.rand(N, generator=g) * 2).cuda()
        T[::7], T[3], T[4] = 0.0, -1.0, float("nan")
        k = torch.randint(-2, 80, (N,), generator=g, dtype=torch.int32).cuda()
        k[5], k[6] = V, V + 5
        p = torch.rand(N, generator=g).cuda() * 1.2
        p[8], p[9], p[10] = 0.0, -1.0, float("nan")
        q = torch.rand(N, generator=g).cuda() * 0.1
        q[11], q[12], q[13] = -1.0, 2.0, float("nan")
        kw = dict(T=T, k=k, p=p, q=q)
        compare(run(z, u, **kw), z, u, **kw)
        compare(run(z, u, T=0.8, k=k), z, u, T=0.8, k=k)
        compare(run(z, u, T=T, p=0.9), z, u, T=T, p=0.9)


@pytest.mark.parametrize("V", [50, 3000, 70000])
def test_ends_of_the_uniform_numbers(V):
    u = torch.tensor([0.0, 1.0, 1 - 2.0 ** -24, 2.0 ** -149, -3.0, 7.0, float("nan"), float("inf"),
                      0.5], device="cuda")
    z, _ = make(9, V, torch.float32, 3, masked=0.3)
    for s in SETTINGS:
        compare(run(z, u, **s), z, u, **s)


def test_infinities_and_nan():
    for V in (40, 5000, 66000):
        z, u = make(8, V, torch.float32, 1)
        z[0] = -math.inf
        z[1, V // 2] = math.nan
        z[2, 3] = math.inf
        z[3, [5, V - 1]] = math.inf
        z[4] = -math.inf
        z[4, V - 1] = -3e38
        z[5, 1:] = -math.inf
        z[6, 0], z[6, 1] = 3e38, -3e38
        z[7] = math.nan
        for s in SETTINGS:
            compare(run(z, u, **s), z, u, **s)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_strides_and_alignment(dt):
    import lm_head_linear_amd as m
    z, u = make(9, 3001, dt, 2)
    wide = torch.full((9, 4000), 50.0, device="cuda").to(dt)
    for s in (dict(), dict(T=0.7, k=30, p=0.9), dict(p=0.9)):
        want = run(z, u, **s)
        for at in (0, 1, 3, 8):
            view = wide[:, at:at + 3001]
            view.copy_(z)
            got = run(view, u, **s)
            assert torch.equal(got.tokens, want.tokens) and torch.equal(got.logp, want.logp)
            wide.fill_(50.0)
    tokens = torch.full((9,), -7, dtype=torch.int64, device="cuda")
    logp = torch.full((9,), -7.0, device="cuda")
    r = m.flce_sample_logits(z, u, tokens=tokens, logp=logp)
    assert r.tokens is tokens and r.logp is logp and bool((tokens >= 0).all())


@pytest.mark.parametrize("V", [37, 4000])
def test_shares_of_the_tokens(V):
    """Uniform numbers on a grid of n: each token is drawn as often as its share of n says,
    to one."""
    n = 20000
    z, _ = make(1, V, torch.float32, 8)
    u = ((torch.arange(n) + 0.5) / n).cuda()
    r = run(z.expand(n, V).contiguous(), u, T=1.5)
    share = torch.softmax(z[0].double() / 1.5, 0).cpu() * n
    count = torch.bincount(r.tokens.cpu(), minlength=V).double()
    assert float((count - share).abs().max()) <= 1.01
    assert bool((r.tokens[1:] >= r.tokens[:-1]).all())


@pytest.mark.parametrize("N,H,V,dt", [(1, 64, 1000, torch.bfloat16), (5, 130, 777, torch.bfloat16),
                                      (48, 256, 3000, torch.bfloat16), (3, 65, 500, torch.float32),
                                      (150, 128, 2000, torch.bfloat16), (20, 33, 515, torch.bfloat16),
                                      (300, 64, 257, torch.float32), (1, 4096, 40000, torch.bfloat16)])
def test_from_the_head(N, H, V, dt):
    """Values on a grid whose products' sums are exact: the logits are the same bits in
    float64, and the tokens those of the oracle."""
    import lm_head_linear_amd as m
    g = torch.Generator().manual_seed(N + V)
    W = (torch.randn(V, H, generator=g) * 16).round().clamp(-255, 255) / 64 / H ** 0.5 * 2
    W = (W * 2 ** 10).round() / 2 ** 10
    h = (torch.randn(N, H, generator=g) * 32).round().clamp(-255, 255) / 32
    W = (W / 2.0 ** -10).round().clamp(-255, 255) * 2.0 ** -10
    z = (h.double() @ W.double().T)
    assert float((h.double().abs() @ W.double().abs().T).max()) < 2 ** 24 * 2.0 ** -15
    u = torch.rand(N, generator=g)
    for s in (dict(), dict(T=0.7, k=20, p=0.9, cap=30.0), dict(T=0.0), dict(p=0.8, q=0.01)):
        r = m.flce_sample(h.to(dt).cuda(), W.to(dt).cuda(), u.cuda(), temperature=s.get("T", 1.0),
                          top_k=s.get("k", 0), top_p=s.get("p", 1.0), min_p=s.get("q", 0.0),
                          softcap=s.get("cap", 0.0))
        compare(r, z, u, **s)


@pytest.mark.parametrize("N,H,V", [(1, 64, 33000), (17, 130, 40001), (33, 64, 32768), (48, 72, 50000),
                                   (64, 65, 32769), (128, 64, 34567), (129, 64, 34567)])
def test_from_a_wide_head(N, H, V):
    """The head's product leaves maxima of each 64 or 128 logits: the tokens are those of the
    logits alone, ties and NaN among them."""
    import lm_head_linear_amd as m
    g = torch.Generator().manual_seed(N + V)
    W = ((torch.randn(V, H, generator=g) * 16).round().clamp(-255, 255) / 64).bfloat16().cuda()
    h = ((torch.randn(N, H, generator=g) * 8).round().clamp(-255, 255) / 32).bfloat16().cuda()
    W[V - 1], W[V // 2] = W[5], W[5]                      # equal logits far apart
    z = (h.double() @ W.double().T).float()
    u = torch.rand(N, generator=g).cuda()
    k = torch.randint(0, 60, (N,), generator=g, dtype=torch.int32).cuda()
    for kw in (dict(top_k=50), dict(temperature=0.0), dict(top_k=k, top_p=0.8, temperature=2.0),
               dict(top_k=1000, softcap=20.0), dict(top_p=0.9), dict(min_p=0.1), dict(top_k=1200)):
        a, b = m.flce_sample(h, W, u, **kw), m.flce_sample_logits(z, u, **kw)
        assert torch.equal(a.tokens, b.tokens) and torch.equal(a.logp, b.logp), kw
    W[7, 3] = float("nan")
    r = m.flce_sample(h, W, u, top_k=5)
    assert bool((r.tokens == -1).all()) and bool(r.logp.isnan().all())
    r = m.flce_sample(torch.zeros_like(h), torch.zeros_like(W), u, top_k=40)   # all equal
    assert bool((r.tokens < 40).all())
    r = m.flce_sample(torch.zeros_like(h), torch.zeros_like(W), u, temperature=0.0)
    assert bool((r.tokens == 0).all())


@pytest.mark.parametrize("N,V,dt", [(1, 56291, torch.bfloat16), (3, 20000, torch.float32),
                                    (64, 16384, torch.bfloat16)])
@pytest.mark.parametrize("k", [100, 130, 500, 1000, 1024, 1025, 2000])
def test_more_ranks_than_parts(N, V, dt, k):
    """Few long rows have the maxima of their parts at hand; a k beyond their number."""
    z, u = make(N, V, dt, V + k)
    for cap in (0.0, 30.0):
        compare(run(z, u, T=1.3, k=k, p=0.7, cap=cap), z, u, T=1.3, k=k, p=0.7, cap=cap)


def test_rows_in_parts_of_the_workspace():
    """More rows than the logits' 512 MiB hold at once: each row is what it is alone."""
    import lm_head_linear_amd as m
    N, H, V = 700, 8, 200000                # 660 rows at a time
    g = torch.Generator(device="cuda").manual_seed(0)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    W = torch.randn(V, H, generator=g, device="cuda").bfloat16()
    u = torch.rand(N, generator=g, device="cuda")
    T = 0.5 + torch.rand(N, generator=g, device="cuda")
    assert m.flce_sample_workspace_size(N, H, V, torch.bfloat16) <= 512 << 20
    r = m.flce_sample(h, W, u, temperature=T, top_k=100)
    for part in (slice(0, 200), slice(600, 700)):
        p = m.flce_sample(h[part].contiguous(), W, u[part].contiguous(),
                          temperature=T[part].contiguous(), top_k=100)
        assert torch.equal(p.tokens, r.tokens[part]) and torch.equal(p.logp, r.logp[part])


def test_captured_streams_and_bits():
    import lm_head_linear_amd as m
    z, u = make(40, 30000, torch.float32, 4)
    T = torch.full((40,), 0.8, device="cuda")
    kw = dict(temperature=T, top_k=50, top_p=0.9)
    want = m.flce_sample_logits(z, u, **kw)
    h, W = torch.randn(4, 64, device="cuda").bfloat16(), torch.randn(999, 64, device="cuda").bfloat16()
    head = m.flce_sample(h, W, u[:4].contiguous(), top_p=0.9)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = m.flce_sample_logits(z, u, **kw)
        ghead = m.flce_sample(h, W, u[:4].contiguous(), top_p=0.9)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.tokens, want.tokens) and torch.equal(got.logp, want.logp)
        assert torch.equal(ghead.tokens, head.tokens) and torch.equal(ghead.logp, head.logp)
        again = m.flce_sample_logits(z, u, **kw)
        assert torch.equal(again.tokens, want.tokens) and torch.equal(again.logp, want.logp)
    outs = []
    for st in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(st):
            outs.append(m.flce_sample_logits(z, u, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(o.tokens, want.tokens) for o in outs)
    # a row does not depend on the others
    one = m.flce_sample_logits(z[7:8], u[7:8], temperature=0.8, top_k=50, top_p=0.9)
    assert int(one.tokens) == int(want.tokens[7]) and float(one.logp) == float(want.logp[7])


def test_decoding_with_a_tied_model():
    """A loop of single tokens: embed, a layer, transform, head, sample; greedy equals the
    best alternative of the log probabilities."""
    import lm_head_linear_amd as m
    torch.manual_seed(1)
    t = m.TiedLMHead(700, 64, transform="gelu", logit_softcapping=30.0, device="cuda",
                     dtype=torch.bfloat16)
    tok = torch.randint(0, 700, (5, 1), device="cuda")
    for i in range(4):
        with torch.no_grad():
            e = t.embed(tok)
            x = torch.tanh(e)
            u = torch.rand(5, 1, device="cuda")
            r = t.sample(x, u, residual=e, temperature=0.0)
            lp = t.logprobs(x, None, residual=e, top_k=1)
            assert torch.equal(r.tokens, lp.top_ids[..., 0])
            nxt = t.sample(x, u, residual=e, temperature=torch.full((5, 1), 0.9, device="cuda"),
                           top_k=30, top_p=0.9, min_p=0.01)
            assert nxt.tokens.shape == (5, 1) and nxt.logp.shape == (5, 1)
            ids = t.logprobs(x, None, residual=e, top_k=30, temperature=0.9).top_ids[:, 0]
            assert bool((ids == nxt.tokens).any(1).all())
            tok = nxt.tokens


def test_no_rows_and_refusals():
    import lm_head_linear_amd as m
    z, u = make(4, 100, torch.float32, 0)
    r = m.flce_sample_logits(z[:0], u[:0])
    assert r.tokens.shape == (0,) and r.logp.shape == (0,)
    W = torch.randn(100, 16, device="cuda").bfloat16()
    assert m.flce_sample(W[:0], W, u[:0]).tokens.shape == (0,)
    for bad in (lambda: m.flce_sample_logits(z.half(), u), lambda: m.flce_sample_logits(z, u[:3]),
                lambda: m.flce_sample_logits(z, u.double()), lambda: m.flce_sample_logits(z.t(), u),
                lambda: m.flce_sample_logits(z, u, top_k=torch.ones(4, device="cuda")),
                lambda: m.flce_sample_logits(z, u, top_p=torch.ones(3, device="cuda")),
                lambda: m.flce_sample_logits(z, u, temperature=torch.ones(4)),
                lambda: m.flce_sample_logits(z, u, top_k=-1),
                lambda: m.flce_sample(W.float(), W, u)):
        with pytest.raises(ValueError):
            bad()
    for bad in (dict(temperature=-1.0), dict(temperature=float("nan")), dict(top_p=0.0),
                dict(top_p=1.5), dict(min_p=-0.1), dict(min_p=1.1), dict(softcap=-1.0),
                dict(temperature=float("inf"))):
        with pytest.raises(m.FlceError):
            m.flce_sample_logits(z, u, **bad)
