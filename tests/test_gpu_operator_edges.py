"""The operators around the head at the ends of their ranges: vocabularies of a few ids,
a vocabulary whose first ids are unreachable, temperatures at which logits differ by
more than float32 holds, more rows than one launch of the norm takes, tables of more than 2^24
ids, batches without a row."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


def make(N, H, V, dt, seed=0):
    """Values on a grid: float32 logits are exact (H 255^2 2^-10 steps below 2^24)."""
    g = torch.Generator().manual_seed(seed)
    q = lambda *s: (torch.randn(*s, generator=g) * 8).round().clamp(-31, 31)  # noqa: E731
    h, W = q(N, H) / 8, q(V, H) / 64
    y = torch.randint(0, V, (N,), generator=g)
    return h.to(dt).cuda(), W.to(dt).cuda(), y.cuda()


@pytest.mark.parametrize("N,dt", [(3, BF), (130, BF), (300, BF), (3, F), (70, F)])
@pytest.mark.parametrize("V", [1, 2, 7, 9])
@pytest.mark.parametrize("H", [1, 16, 24])
def test_a_vocabulary_of_a_few_ids(N, dt, V, H):
    import lm_head_linear_amd as m
    h, W, y = make(N, H, V, dt, seed=V)
    y[0] = -100
    g = torch.Generator().manual_seed(1)
    a, b = torch.randn(N, generator=g).cuda(), torch.randn(N, generator=g).cuda()
    r = m.flce_logprobs(h, W, y, top_k=3, temperature=0.8)
    x = h.double() @ W.double().t() / 0.8
    lp = torch.log_softmax(x, 1)
    live = y != -100
    at = y.clamp_min(0)[:, None]
    ent = -(lp.exp() * lp).sum(1)
    # as in test_gpu_logprobs: |x| < 2^7 here
    tol = 2.0 ** -18 + 2.0 ** -14
    assert float((r.logp - lp.gather(1, at)[:, 0] * live).abs().max()) < tol
    assert float((r.entropy - ent * live).abs().max()) < 40 * tol
    k = min(3, V)
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.top_ids[live][:, :k], ids[live]) and bool((r.top_ids[:, k:] == -1).all())
    dH, dW = m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b, temperature=0.8)
    hot = torch.zeros_like(x).scatter_(1, at, 1.0)
    G = a[:, None] * (hot - lp.exp()) - b[:, None] * lp.exp() * (lp + ent[:, None])
    G = G * live[:, None] / 0.8
    # G errs by the logits' and the lse's rounding (|x| < 2^6: 2^-17) in each of its terms, which
    # cancel where one id holds all; by the entropy's error (2^-14); and bf16 by half a step
    # of itself. Stored gradients by half a step.
    mag = a.abs()[:, None] * (hot + lp.exp()) + b.abs()[:, None] * lp.exp() * ((lp + ent[:, None]).abs() + 1)
    dG = 2.0 ** -13 * mag * live[:, None] / 0.8 + (2.0 ** -8 * G.abs() if dt == BF else 0)
    for got, ref, err in ((dH, G @ W.double(), dG @ W.double().abs()),
                          (dW, G.t() @ h.double(), dG.t() @ h.double().abs())):
        off = (got.double() - ref).abs()
        assert bool((off <= err + torch.finfo(dt).eps * ref.abs()).all()), float((off - err).max())


@pytest.mark.parametrize("K", [1, 5, 20])
@pytest.mark.parametrize("N", [60, 300, 1100])
@pytest.mark.parametrize("reach", [69997, 40000, 100])
def test_the_first_ids_are_unreachable(K, N, reach):
    """-inf logits in all tiles that would bound the others; `reach` ids are left, the
    last ones, fewer than the alternatives at the far end."""
    import lm_head_linear_amd as m
    V = 70000
    h, W, y = make(N, 16, V, BF, seed=K)
    h[:, 0], W[:, 0] = 1, 0
    W[:V - reach, 0] = -torch.inf
    y = y % reach + V - reach
    r = m.flce_logprobs(h, W, y, top_k=K)
    x = h.float() @ W.float().t()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(r.top_ids, order)
    lp = torch.log_softmax(x.double(), 1)
    assert float((r.logp - lp.gather(1, y[:, None])[:, 0]).abs().max()) < 2.0 ** -14
    W[:V - 3, 0] = -torch.inf
    r = m.flce_logprobs(h, W, None, top_k=K)
    k = min(K, 3)
    assert bool((r.top_ids[:, :k] >= V - 3).all()) and bool((r.top_ids[:, k:] == -1).all())


@pytest.mark.parametrize("N,dt", [(3, BF), (150, BF), (3, F)])
@pytest.mark.parametrize("T", [1e-30, 1e-37, 1e30])
@pytest.mark.parametrize("V", [300, 20000])
def test_temperatures_far_from_one(N, dt, T, V):
    """Near 0 the best tokens share the probability; far above, all do."""
    import lm_head_linear_amd as m
    h, W, y = make(N, 16, V, dt, seed=4)
    # logits of -32 to 32: divided by 1e-37 they are in float32's range, some differences not
    h[:, 0], h[:, 1:], W[:, 0] = 1, 0, (W[:, 0] * 64).clamp(-32, 32)
    W[::5, 0], W[V // 2:, 0] = 32, -32
    r = m.flce_logprobs(h, W, y, temperature=T, top_k=2)
    z = h.float() @ W.float().t()
    best = z == z.max(1, keepdim=True).values
    n = best.sum(1).double() if T < 1 else torch.full((N,), float(V), device="cuda").double()
    assert float((r.entropy.double() - n.log()).abs().max()) < 1e-4
    given = best.gather(1, y[:, None])[:, 0] if T < 1 else torch.ones_like(y, dtype=torch.bool)
    assert float((r.logp.double() + n.log())[given].abs().sum()) < 1e-4 * N
    assert bool((r.logp[~given] < -1e20).all())
    assert float((r.top_logp[:, 0].double() + n.log()).abs().max()) < 1e-4


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("residual", [False, True])
def test_more_rows_than_a_launch_of_the_norm(dt, residual):
    import lm_head_linear_amd as m
    N, H = (1 << 21) + 300, 6
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(N, H, generator=g, device="cuda").to(dt)
    r = torch.randn(N, H, generator=g, device="cuda").to(dt) if residual else None
    w = torch.rand(H, generator=g, device="cuda").to(dt)
    y, s, q = m.flce_rms_norm(x, w, r)
    v = s.double()
    rstd = 1 / ((v * v).mean(1) + 1e-6).sqrt()
    assert float((q.double() / rstd - 1).abs().max()) < 2.0 ** -20
    want = v * rstd[:, None] * w.double()
    assert bool(((y.double() - want).abs() <= (torch.finfo(dt).eps / 2 + 2.0 ** -20) * want.abs()).all())
    dx, dw = m.flce_rms_norm_backward(y, s, w, q)
    n, gy = v * rstd[:, None], y.double() * w.double()
    dx_ref = rstd[:, None] * (gy - n * (gy * n).mean(1, keepdim=True))
    mag = rstd[:, None] * (gy.abs() + n.abs() * (gy * n).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - dx_ref).abs() <= torch.finfo(dt).eps / 2 * dx_ref.abs()
                 + 2.0 ** -19 * mag).all())
    terms = y.double() * n
    # float32 sums in chains of N / 16384 rows and 25 more (rows of 6 share a workgroup)
    chain = (N / 16384 + 95) * 2.0 ** -24
    assert bool(((dw.double() - terms.sum(0)).abs() <= torch.finfo(dt).eps / 2 * terms.sum(0).abs()
                 + chain * terms.abs().sum(0)).all())


@pytest.mark.parametrize("N", [700, 40000])
def test_a_table_of_more_than_2_24_ids(N):
    import lm_head_linear_amd as m
    V, H = (1 << 24) + 77, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    t = torch.randint(V - 500, V, (N,), generator=g, device="cuda")
    t[::2] = torch.randint(0, V, (t[::2].numel(),), generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda").bfloat16()
    assert torch.equal(m.flce_embedding(t, W), W[t])
    # whole numbers of at most 8 bits: sums are exact in float32
    d = torch.randint(-9, 10, (N, H), generator=g, device="cuda").bfloat16()
    want = torch.zeros(V, H, device="cuda").index_add(0, t, d.float())
    got = m.flce_embedding_backward(t, d, V, grad_dtype=F)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("shape", [(0,), (0, 5), (3, 0)])
def test_a_batch_without_a_row(dt, shape):
    import lm_head_linear_amd as m
    t = m.TiedLMHead(50, 16, device="cuda", dtype=dt)
    x = torch.zeros(shape, dtype=torch.int64, device="cuda")
    e = t.embed(x)
    r = t.logprobs(torch.tanh(e), x, residual=e, top_k=2)
    assert r.logp.shape == shape and r.top_ids.shape == (*shape, 2)
    (r.logp.sum() + r.entropy.sum()).backward()
    assert not bool(t.weight.grad.any()) and not bool(t.norm_weight.grad.any())
    assert t.logprobs(e).lse.shape == shape and math.prod(shape) == 0
