"""The operators around the head as they are used together: a small model whose
embedding and head share one table (TiedLMHead), trained on the head's loss and on
token log probabilities, and the same step made of the plain calls with the table's
two gradients added in place.

Tolerances: the float32 chain against the same formulas in float64: every stored value
is off by a few roundings of its terms (u = 2^-24, rows of at most 48 terms, tables of
300 rows); 2e-5 of the largest value leaves a factor of ten. bf16: each of the stages
rounds its rows to 2^-8 of themselves and the gradients are those of the rounded rows,
so the check is bit equality between the module and the calls it is made of."""
import pytest
import torch

pytestmark = pytest.mark.gpu
IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


def head(dt, **kw):
    import lm_head_linear_amd as m
    torch.manual_seed(4)
    t = m.TiedLMHead(300, 48, embed_scale=48 ** 0.5, norm_eps=1e-5, device="cuda", dtype=dt, **kw)
    with torch.no_grad():
        t.weight.mul_(4)
        t.norm_weight.add_(0.2 * torch.randn(48, device="cuda").to(dt))
    return t


def batch():
    g = torch.Generator().manual_seed(9)
    x = torch.randint(0, 300, (2, 70), generator=g)
    x[0, :5] = IGN                            # padding in front
    y = torch.randint(0, 300, (2, 70), generator=g)
    y[:, -3:] = IGN
    y[0, :5] = IGN
    return x.cuda(), y.cuda()


def reference(W, nw, x, y, mix, eps, cap, offset=0.0):
    """The forward in float64 from elementary operations."""
    e = W[x.clamp_min(0)] * 48 ** 0.5 * (x != IGN)[..., None]
    s = e + torch.tanh(e) * mix
    h = s / ((s * s).mean(-1, keepdim=True) + eps).sqrt() * (nw + offset)
    z = h @ W.t()
    if cap:
        z = cap * torch.tanh(z / cap)
    lp = z - torch.logsumexp(z, -1, keepdim=True)
    live = y != IGN
    return lp, live, lp.gather(-1, y.clamp_min(0)[..., None])[..., 0] * live


@pytest.mark.parametrize("what", ["loss", "logprobs"])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_a_training_step_in_float32(what, cap):
    t = head(torch.float32, logit_softcapping=cap, reduction="mean")
    x, y = batch()
    mix, c = torch.randn(2, 70, 48, device="cuda"), torch.randn(2, 70, device="cuda")
    W, nw = (p.detach().double().requires_grad_() for p in (t.weight, t.norm_weight))
    lp, live, ref = reference(W, nw, x, y, mix.double(), 1e-5, cap)
    e = t.embed(x)
    if what == "loss":
        out = t.loss(torch.tanh(e) * mix, y, residual=e)
        want = -ref.sum() / live.sum()
    else:
        r = t.logprobs(torch.tanh(e) * mix, y, residual=e, top_k=3)
        out = (r.logp * c).sum() + 0.1 * r.entropy.sum()
        ent = -(lp.exp() * lp).sum(-1) * live
        want = (ref * c.double()).sum() + 0.1 * ent.sum()
        assert float((r.logp.detach().double() - ref.detach()).abs().max()) < 1e-5
        order = torch.sort(lp, dim=-1, descending=True).values[..., :3]
        assert float((r.top_logp.detach()[live].double() - order.detach()[live]).abs().max()) < 1e-5
    out.backward()
    want.backward()
    got, ref = float(out.detach()), float(want.detach())
    assert abs(got - ref) < 2e-5 * max(1.0, abs(ref))
    for got, ref in ((t.weight.grad, W.grad), (t.norm_weight.grad, nw.grad)):
        assert float((got.double() - ref).abs().max()) < 2e-5 * float(ref.abs().max())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_the_calls_of_a_step_by_hand(dt):
    """Log probabilities and their gradients by the plain calls, the embedding's
    gradient added to the head's table in place."""
    import lm_head_linear_amd as m
    t = head(dt)
    x, y = batch()
    W, nw = t.weight.detach(), t.norm_weight.detach()
    flat, yf = x.reshape(-1), y.reshape(-1)
    a, b = torch.randn(140, device="cuda"), 0.1 * torch.randn(140, device="cuda")
    scale = 48 ** 0.5
    e = m.flce_embedding(flat, W, scale=scale, padding_index=IGN)
    h, s, rstd = m.flce_rms_norm(torch.tanh(e), nw, e, eps=1e-5)
    r = m.flce_logprobs(h, W, yf)
    dH, dW = m.flce_logprobs_backward(h, W, yf, r.lse, r.entropy, a, b)
    head_only = dW.clone()
    ds, dnw = m.flce_rms_norm_backward(dH, s, nw, rstd)
    de = (ds.float() + ds.float() * (1 - torch.tanh(e).float() ** 2)).to(dt)
    m.flce_embedding_backward(flat, de, 300, scale=scale, padding_index=IGN, dW=dW,
                              accumulate_dW=True)
    # the module on the same rows: the norm's and the head's parts bit for bit
    e2 = e.detach().requires_grad_()
    r2 = t.logprobs(torch.tanh(e2), yf, residual=e2)
    assert torch.equal(r2.logp, r.logp) and torch.equal(r2.entropy, r.entropy)
    ((r2.logp * a).sum() + (r2.entropy * b).sum()).backward()
    assert torch.equal(t.weight.grad, head_only) and torch.equal(t.norm_weight.grad, dnw)
    emb = m.flce_embedding_backward(flat, de, 300, scale=scale, padding_index=IGN,
                                    grad_dtype=torch.float32)
    want = head_only.double() + emb.double()
    tol = torch.finfo(dt).eps / 2 * want.abs() * (1 + 2.0 ** -6) + 2.0 ** -22 * emb.abs().max()
    assert bool(((dW.double() - want).abs() <= tol).all())


def test_decoding_one_token_at_a_time():
    """Rows of a longer batch give the bits of the whole batch: the few-token kernel has
    one order of sums for any count of rows up to 128."""
    t = head(torch.bfloat16)
    x, y = batch()
    with torch.no_grad():
        e = t.embed(x)
        whole = t.logprobs(torch.tanh(e)[0], y[0], residual=e[0], top_k=4)
        for i in (0, 6, 69):
            one = t.logprobs(torch.tanh(e)[0, i:i + 1], y[0, i:i + 1], residual=e[0, i:i + 1], top_k=4)
            assert torch.equal(one.top_ids[0], whole.top_ids[i])
            assert torch.equal(one.top_logp[0], whole.top_logp[i])
            assert torch.equal(one.logp[0], whole.logp[i])
        last = t.logprobs(torch.tanh(e)[:, -1], residual=e[:, -1], top_k=2)   # strided rows
        assert last.logp is None and last.top_ids.shape == (2, 2)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_slice_of_odd_rows(dt):
    """Rows from the middle of a batch of odd width start at any element."""
    import lm_head_linear_amd as m
    torch.manual_seed(2)
    W = (0.1 * torch.randn(700, 37, device="cuda")).to(dt)
    x = torch.randn(9, 37, device="cuda").to(dt).requires_grad_()
    y = torch.randint(0, 700, (9,), device="cuda")
    a = m.token_logprobs(x[2:7], y[2:7], W, top_k=2)
    b = m.token_logprobs(x[2:7].clone(), y[2:7].clone(), W, top_k=2)
    assert torch.equal(a.logp, b.logp) and torch.equal(a.top_ids, b.top_ids)
    (g,) = torch.autograd.grad(a.logp.sum(), x)
    (h,) = torch.autograd.grad(b.logp.sum(), x)
    assert torch.equal(g, h) and not bool(g[:2].any()) and bool(g[2:7].any())


def test_two_streams_at_once():
    """The same calls on two streams, each with workspaces of its own, and one of them
    made current only for the call."""
    import lm_head_linear_amd as m
    torch.manual_seed(1)
    W = (0.1 * torch.randn(5000, 256, device="cuda")).bfloat16()
    jobs = []
    for n in (3, 200):
        h = torch.randn(n, 256, device="cuda").bfloat16()
        y = torch.randint(0, 5000, (n,), device="cuda")
        a = torch.randn(n, device="cuda")
        jobs.append((h, y, a))

    def step(h, y, a):
        r = m.flce_logprobs(h, W, y, top_k=3)
        dH, dW = m.flce_logprobs_backward(h, W, y, r.lse, None, a)
        m.flce_embedding_backward(y, dH, 5000, dW=dW, accumulate_dW=True)
        n, s, q = m.flce_rms_norm(dH, W[0])
        return [r.logp, r.top_ids, dH, dW, n, q]
    want = [step(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*jobs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(g, want[i]))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_captured_training_step(dt):
    """Embedding, norm, loss, log probabilities and all their gradients in one graph,
    recorded with no eager autograd graph of the parameters alive."""
    t = head(dt)
    x, y = batch()
    c = torch.randn(2, 70, device="cuda")

    def step():
        e = t.embed(x)
        loss = t.loss(torch.tanh(e), y, residual=e)
        r = t.logprobs(torch.tanh(e), y, residual=e, top_k=3)
        out = loss + (r.logp * c).sum()
        out.backward()
        return out.detach(), r.top_ids, r.lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            t.zero_grad(set_to_none=True)
            want = [v.clone() for v in step()] + [p.grad.clone() for p in t.parameters()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    t.zero_grad(set_to_none=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    got = [*outs, *(p.grad for p in t.parameters())]
    for _ in range(3):
        for v in got:
            v.fill_(7)
        torch.randn(300, 300, device="cuda").sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_with_one_workspace():
    """Graphs of different calls that share their workspace, replayed in turn."""
    import lm_head_linear_amd as m
    torch.manual_seed(6)
    W = (0.1 * torch.randn(3000, 64, device="cuda")).bfloat16()
    need = max(m.flce_logprobs_workspace_size(n, 64, 3000, torch.bfloat16, 9) for n in (12, 300))
    need = max(need, m.flce_embedding_backward_workspace_size(300, 64, 3000))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    jobs = []
    for n in (12, 300):
        h = torch.randn(n, 64, device="cuda").bfloat16()
        y = torch.randint(0, 3000, (n,), device="cuda")
        r = m.flce_logprobs(h, W, y, top_k=9, workspace=ws)
        dW = m.flce_embedding_backward(y, h, 3000, workspace=ws)
        kw = dict(logp=r.logp, entropy=r.entropy, lse=r.lse, top_logp=r.top_logp,
                  top_ids=r.top_ids)
        torch.cuda.synchronize()
        want = [v.clone() for v in (*r, dW)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.flce_logprobs(h, W, y, top_k=9, workspace=ws, **kw)
            m.flce_embedding_backward(y, h, 3000, dW=dW, workspace=ws)
        jobs.append((g, [*r, dW], want, (h, y)))
    for _ in range(3):
        for g, got, want, _ in jobs:
            for v in got:
                v.fill_(5)
            g.replay()
        torch.cuda.synchronize()
        for g, got, want, _ in jobs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
