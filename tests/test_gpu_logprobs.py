"""Token log probabilities, entropy and top alternatives, forward and backward,
against the definitions in float64.

The inputs lie on a grid (see grid): every product and partial sum of a logit is
a whole number of steps below 2^24, so the float32 logits of any kernel are exact
and the ranking, ties included, is that of the float64 logits.

Tolerances, forward: with exact logits the scalars err by the hardware exp2's
argument (z log2 e - m log2 e, rounded: u |z| log2 e each, u = 2^-24), the sums
(below 2^-19 relative, from chains of at most 100 additions and joins) and the
logarithm. log S is off by the relative error of S, at most 2^-18 with |z| < 16;
logp and lse add u (|x| + |M|). With a softcap s, x itself is off by 1e-6 s / T
(tanh from the hardware exp2 and reciprocal, as in logits_tolerance), which also
enters every exponent. The entropy weighs those errors by |x - M|, at most 40 here.
Backward: G errs by those relative errors (float32) and half a bf16 step (bf16);
stored gradients by half a step of their type. The bf16 bound is that of the head's
own gradients (2e-2 of the largest), the float32 one 1e-4."""
import math

import pytest
import torch

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


def grid(x, step):
    return (x / step).round().clamp(-255, 255) * step


def make(N, H, V, dt, seed=0, ignored=0.2, peaked=True):
    g = torch.Generator().manual_seed(1000 + seed)
    std = 1.28 / math.sqrt(H)
    W = grid(std * torch.randn(V, H, generator=g), 2.0 ** math.floor(math.log2(std / 32)))
    y = torch.randint(0, V, (N,), generator=g)
    h = torch.randn(N, H, generator=g)
    if peaked:
        h = h + 12 * torch.rand(N, 1, generator=g) / (H * std * std) * W[y]
    h = grid(h, 2.0 ** -5)
    if N > 2:
        y[torch.randperm(N, generator=g)[: int(ignored * N)]] = IGN
    a, b = torch.randn(N, generator=g), 0.3 * torch.randn(N, generator=g)
    return [t.cuda() for t in (h.to(dt), W.to(dt), y, a, b)]


def reference(h, W, y, K, cap, T, a=None, b=None):
    """On the GPU in float64 (float32 logits of grid inputs are exact as well)."""
    z = h.double() @ W.double().t()
    x = (cap * torch.tanh(z / cap) if cap else z) / T
    lse = torch.logsumexp(x, 1)
    lp = x - lse[:, None]
    p = lp.exp()
    live = torch.ones_like(lse, dtype=torch.bool) if y is None else y != IGN
    ent = -(p * lp).sum(1)
    out = dict(lse=lse * live, entropy=ent * live, live=live, z=z)
    if y is not None:
        at = y.clamp_min(0)[:, None]
        out["logp"] = lp.gather(1, at)[:, 0] * live
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :K]
    out["top_ids"] = torch.where(live[:, None], order, -1)
    out["top_logp"] = lp.gather(1, order).masked_fill(~live[:, None], -math.inf)
    if a is not None or b is not None:
        a, b = (torch.zeros_like(lse) if t is None else t.double() for t in (a, b))
        hot = torch.zeros_like(p).scatter_(1, at, 1.0)
        G = a[:, None] * (hot - p) - b[:, None] * p * (lp + ent[:, None])
        if cap:
            G = G * (1 - torch.tanh(z / cap) ** 2)
        G = G * live[:, None] / T
        out["dH"], out["dW"] = G @ W.double(), G.t() @ h.double()
    return out


def check_forward(r, ref, K, cap, T):
    V = ref["z"].shape[1]
    tol = 2.0 ** -18 + 32 * U / T * 4 + 2e-6 * cap / T
    live = ref["live"]

    def close(got, want, t):
        d = (got.double() - want).abs()
        assert not bool((d > t).any()), (float(d.max()), t)
    close(r.lse, ref["lse"], tol)
    close(r.entropy, ref["entropy"], 40 / T * tol)
    if r.logp is not None:
        close(r.logp, ref["logp"], tol)
        assert bool((r.logp[~live] == 0).all())
    assert bool((r.lse[~live] == 0).all()) and bool((r.entropy[~live] == 0).all())
    k = min(K, V)
    assert torch.equal(r.top_ids[:, :k], ref["top_ids"][:, :k])
    assert bool((r.top_ids[:, k:] == -1).all()) and bool((r.top_logp[:, k:] == -math.inf).all())
    if k:
        close(r.top_logp[live][:, :k], ref["top_logp"][live][:, :k], tol)
        assert bool((r.top_logp[~live] == -math.inf).all())


BF, F = torch.bfloat16, torch.float32
# few tokens (three widths of the kernel, its odd rows and short vocabularies), the
# matrix-core tiles (one and several of each edge, gathered, odd H), float32
FORWARD = [(1, 64, 1, BF, 3), (1, 4096, 5000, BF, 8), (2, 33, 63, BF, 32), (15, 100, 64, BF, 4),
           (16, 1024, 4097, BF, 1), (17, 257, 1000, BF, 20), (33, 96, 70000, BF, 5),
           (64, 512, 999, BF, 32), (65, 512, 999, BF, 10), (65, 41, 130, BF, 32), (40, 130, 515, BF, 4),
           (128, 258, 1001, BF, 3), (100, 385, 333, BF, 17), (129, 512, 999, BF, 10),
           (140, 41, 130, BF, 32),
           (200, 64, 9000, BF, 9), (150, 64, 5000, BF, 17), (600, 72, 40000, BF, 20),
           (200, 64, 20000, BF, 12), (140, 64, 70000, BF, 32),
           (300, 136, 2000, BF, 7), (513, 72, 255, BF, 3), (700, 520, 3001, BF, 0),
           (3, 1, 70, BF, 2), (130, 3, 300, BF, 5), (5, 1, 70, F, 2),
           (1, 64, 1, F, 2), (3, 77, 200, F, 6), (64, 33, 64, F, 20), (65, 515, 1001, F, 32),
           (257, 130, 333, F, 0)]


@pytest.mark.parametrize("N,H,V,dt,K", FORWARD)
@pytest.mark.parametrize("cap,T", [(0.0, 1.0), (30.0, 0.7)])
def test_forward(N, H, V, dt, K, cap, T):
    import lm_head_linear_amd as m
    h, W, y, _, _ = make(N, H, V, dt, seed=N + V)
    kw = dict(softcap=cap, temperature=T, top_k=K)
    st = torch.full((), -1, dtype=torch.int32, device="cuda")
    r = m.flce_logprobs(h, W, y, status=st, **kw)
    check_forward(r, reference(h, W, y, K, cap, T), K, cap, T)
    assert int(st) == 0
    again = m.flce_logprobs(h, W, y, **kw)
    assert all(torch.equal(a, b) for a, b in zip(r, again))
    free = m.flce_logprobs(h, W, None, **kw)
    assert free.logp is None
    check_forward(free, reference(h, W, None, K, cap, T), K, cap, T)


@pytest.mark.parametrize("N,H,V,dt,K", [(7, 64, 900, BF, 32), (150, 64, 900, BF, 32),
                                        (150, 64, 900, F, 32), (9, 64, 900, F, 32)])
def test_ties_go_to_the_lowest_id(N, H, V, dt, K):
    """Every logit repeated across lists, tiles and threads; a row of equal logits."""
    import lm_head_linear_amd as m
    h, W, y, _, _ = make(N, H, V, dt, ignored=0.0)
    W = W[torch.arange(V, device="cuda") % 11].contiguous()
    h[3] = 0
    r = m.flce_logprobs(h, W, y, top_k=K)
    ref = reference(h, W, y, K, 0.0, 1.0)
    assert torch.equal(r.top_ids, ref["top_ids"])
    assert r.top_ids[3].tolist() == list(range(K))


@pytest.mark.parametrize("K", [1, 5, 9, 32])
@pytest.mark.parametrize("order", ["rising", "falling", "flat"])
def test_alternatives_wherever_they_are(K, order):
    """A vocabulary large enough that its first tiles bound the rest: logits that rise
    with the id (the bound holds nothing back and every list is full), that fall (the
    rest is empty), and that do neither."""
    import lm_head_linear_amd as m
    N, H, V = 300, 64, 70000
    h, W, y, _, _ = make(N, H, V, BF, seed=3)
    step = (torch.arange(V, device="cuda") // 512).float() * 2.0 ** -3
    W[:, 0] = (step if order == "rising" else -step if order == "falling" else 0 * step).to(BF)
    h[:, 0] = 1
    r = m.flce_logprobs(h, W, y, top_k=K)
    ref = reference(h, W, y, K, 0.0, 1.0)
    assert torch.equal(r.top_ids, ref["top_ids"])
    live = ref["live"]
    assert float((r.top_logp[live].double() - ref["top_logp"][live]).abs().max()) < 1e-4
    again = m.flce_logprobs(h, W, y, top_k=K)
    assert all(torch.equal(a, b) for a, b in zip(r, again))


@pytest.mark.parametrize("N", [5, 130])
@pytest.mark.parametrize("dt", [BF, F])
def test_infinite_and_nan_rows(N, dt):
    import lm_head_linear_amd as m
    V, H, K = 700, 64, 9
    h, W, y, _, _ = make(N, H, V, dt, ignored=0.0)
    W[:, 0] = 1.0
    h[:, 0] = 0
    clean = m.flce_logprobs(h, W, y, top_k=K)
    W2 = W.clone()
    W2[100:, 1] = float("-inf")             # most of the vocabulary unreachable
    h2 = h.clone()
    h2[:, 1] = 1.0
    y2 = y.clamp_max(99)
    r = m.flce_logprobs(h2, W2, y2, top_k=K)
    ref = reference(h2, W2[:100], y2, K, 0.0, 1.0)
    assert torch.equal(r.top_ids, ref["top_ids"])
    assert float((r.logp.double() - ref["logp"]).abs().max()) < 1e-4
    assert float((r.entropy.double() - ref["entropy"]).abs().max()) < 1e-3
    W2[5:, 1] = float("-inf")               # fewer left than are asked for
    r = m.flce_logprobs(h2, W2, y2.clamp_max(4), top_k=K)
    assert bool((r.top_ids[:, 5:] == -1).all()) and bool((r.top_ids[:, :5].sort(1).values == torch.arange(5, device="cuda")).all())
    h3 = h.clone()
    h3[2] = float("nan")                    # one row only
    r = m.flce_logprobs(h3, W, y, top_k=K)
    keep = torch.arange(N, device="cuda") != 2
    assert bool(r.logp[2].isnan()) and bool(r.entropy[2].isnan())
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(r, clean))


@pytest.mark.parametrize("N", [6, 90])
@pytest.mark.parametrize("dt", [BF, F])
def test_bad_tokens(N, dt):
    import lm_head_linear_amd as m
    h, W, y, a, b = make(N, 64, 300, dt, ignored=0.3)
    y[0], y[1] = 300, -5
    ok = y.clone()
    ok[:2] = 0
    st = torch.full((), -1, dtype=torch.int32, device="cuda")
    r = m.flce_logprobs(h, W, y, top_k=4, status=st)
    good = m.flce_logprobs(h, W, ok, top_k=4)
    assert int(st) == 5 and bool(r.logp[:2].isnan().all())
    assert torch.equal(r.logp[2:], good.logp[2:])
    assert all(torch.equal(x, z) for x, z in zip(r[1:], good[1:]))
    st.fill_(-1)
    dH, dW = m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b, status=st)
    assert int(st) == 5 and bool(dH[:2].isnan().all()) and bool(dW.isnan().all())
    assert not bool(dH[2:].isnan().any())


@pytest.mark.parametrize("N", [4, 80])
def test_every_row_ignored_and_none(N):
    import lm_head_linear_amd as m
    h, W, y, a, b = make(N, 64, 300, BF)
    y[:] = IGN
    r = m.flce_logprobs(h, W, y, top_k=2)
    assert not any(bool(t.any()) for t in r[:3]) and bool((r.top_ids == -1).all())
    dH, dW = m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b)
    assert not bool(dH.any()) and not bool(dW.any())
    r = m.flce_logprobs(h[:0], W, y[:0], top_k=2)
    assert r.logp.shape == (0,) and r.top_ids.shape == (0, 2)
    dW = torch.ones_like(W)
    m.flce_logprobs_backward(h[:0], W, y[:0], r.lse, r.entropy, a[:0], b[:0], dW=dW,
                             accumulate_dW=True)
    assert bool((dW == 1).all())
    m.flce_logprobs_backward(h[:0], W, y[:0], r.lse, r.entropy, a[:0], b[:0], dW=dW)
    assert not bool(dW.any())


BACKWARD = [(1, 64, 300, BF), (17, 200, 3000, BF), (40, 128, 1000, BF), (128, 133, 700, BF),
            (129, 264, 1100, BF), (300, 136, 2000, BF), (700, 133, 1500, BF),
            (1, 33, 300, F), (70, 130, 515, F), (300, 64, 1000, F)]


@pytest.mark.parametrize("N,H,V,dt", BACKWARD)
@pytest.mark.parametrize("cap,T", [(0.0, 1.0), (30.0, 1.3)])
@pytest.mark.parametrize("parts", ["both", "logp", "entropy"])
def test_backward(N, H, V, dt, cap, T, parts, monkeypatch):
    import lm_head_linear_amd as m
    monkeypatch.setenv("FLCE_VCHUNK", "512")        # several chunks of the vocabulary
    h, W, y, a, b = make(N, H, V, dt, seed=7)
    a, b = (a if parts != "entropy" else None), (b if parts != "logp" else None)
    kw = dict(softcap=cap, temperature=T)
    r = m.flce_logprobs(h, W, y, **kw)
    dH, dW = m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b, **kw)
    ref = reference(h, W, y, 0, cap, T, a, b)
    tol = gu.GRAD_TOL[dt]
    gu.assert_grad("dH", dH, ref["dH"].cpu().numpy(), tol)
    gu.assert_grad("dW", dW, ref["dW"].cpu().numpy(), tol)
    assert not bool(dH[y == IGN].any())
    again = m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b, **kw)
    assert torch.equal(dH, again[0]) and torch.equal(dW, again[1])
    base = (0.1 * torch.randn(V, H, device="cuda")).to(dt)
    acc = base.clone()
    m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b, dW=acc, accumulate_dW=True, **kw)
    gu.assert_grad("dW added", acc, (ref["dW"] + base.double()).cpu().numpy(), tol)
    if dt == BF:
        eH, eW = m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b,
                                          grad_dtype=torch.float32, **kw)
        gu.assert_grad("dH f32", eH, ref["dH"].cpu().numpy(), 1e-4)
        gu.assert_grad("dW f32", eW, ref["dW"].cpu().numpy(), 1e-4)


@pytest.mark.parametrize("N,H", [(5, 72), (129, 136), (300, 133), (800, 600), (1500, 64)])
@pytest.mark.parametrize("chunk", ["0", "4096"])
def test_backward_with_split_dH(N, H, chunk, monkeypatch):
    """dH summed from many segments of a chunk's vocabulary, of one chunk and of three,
    the last of which leaves segments empty."""
    import lm_head_linear_amd as m
    monkeypatch.setenv("FLCE_VCHUNK", chunk)
    h, W, y, a, b = make(N, H, 9000, BF, seed=8)
    r = m.flce_logprobs(h, W, y)
    need = m.flce_logprobs_backward_workspace_size(N, H, 9000, BF)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    dH, dW = m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b, workspace=ws)
    ref = reference(h, W, y, 0, 0.0, 1.0, a, b)
    gu.assert_grad("dH", dH, ref["dH"].cpu().numpy(), gu.GRAD_TOL[BF])
    gu.assert_grad("dW", dW, ref["dW"].cpu().numpy(), gu.GRAD_TOL[BF])
    again = m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b)
    assert torch.equal(dH, again[0]) and torch.equal(dW, again[1])


@pytest.mark.parametrize("H", [128, 133])
@pytest.mark.parametrize("accumulate", [False, True])
def test_a_row_whose_terms_cancel(H, accumulate, monkeypatch):
    """300 pairs of rows with one token and upstream gradients a and -a (1 - 2^-8): the
    token's dW row is 2^-8 of its terms, below what a bf16 G resolves of them. It has
    to be right to a few steps of its own: G errs by exp's 2^-18 of the terms, 2^-10 of
    the row, the other tokens' G by 2^-9 p of the terms with p < 2^-5 (2^-6 of the row)
    with random signs over 600 rows, and the row is rounded twice (2^-8 each)."""
    import lm_head_linear_amd as m
    monkeypatch.setenv("FLCE_VCHUNK", "512")
    h, W, y, a, _ = make(300, H, 1200, BF, ignored=0.0, peaked=False)
    h = h.repeat(2, 1)
    y = torch.full((600,), 700, device="cuda")
    a = a.abs() + 0.5
    a = torch.cat([a, -a * (1 - 2.0 ** -8)])
    r = m.flce_logprobs(h, W, y)
    base = torch.zeros_like(W)
    _, dW = m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, dW=base if accumulate else None,
                                     accumulate_dW=accumulate)
    ref = reference(h, W, y, 0, 0.0, 1.0, a, None)["dW"][700]
    err = (dW[700].double() - ref).norm() / ref.norm()
    assert float(err) < 2.0 ** -6, float(err)


@pytest.mark.parametrize("N,H,V", [(1, 64, 300), (9, 72, 1100), (30, 65, 1001), (60, 64, 1003),
                                   (100, 72, 997), (300, 72, 1001)])
def test_what_the_workspace_held_does_not_matter(N, H, V, monkeypatch):
    """Workspaces full of NaN bit patterns give the same bits as zeroed ones."""
    import lm_head_linear_amd as m
    monkeypatch.setenv("FLCE_VCHUNK", "512")
    h, W, y, a, b = make(N, H, V, BF)
    ws = torch.empty(m.flce_logprobs_workspace_size(N, H, V, BF, 6), dtype=torch.uint8, device="cuda")
    wb = torch.empty(m.flce_logprobs_backward_workspace_size(N, H, V, BF), dtype=torch.uint8,
                     device="cuda")
    got = []
    for byte in (0, 255):
        ws.fill_(byte), wb.fill_(byte)
        r = m.flce_logprobs(h, W, y, top_k=6, workspace=ws)
        got.append([*r, *m.flce_logprobs_backward(h, W, y, r.lse, r.entropy, a, b, workspace=wb)])
    assert all(torch.equal(p, q) for p, q in zip(*got))


def test_gradients_against_differences():
    """Autograd of the float32 form against central differences of its forward in
    random directions: a step of 2^-7 (directions of norm 1) has a truncation
    error of order 2^-14 and a rounding error of some 40 u / 2^-7."""
    import lm_head_linear_amd as m
    torch.manual_seed(5)
    h = torch.randn(2, 3, 12, device="cuda", requires_grad=True)
    W = torch.randn(30, 12, device="cuda", requires_grad=True)
    y = torch.tensor([[3, IGN, 29], [0, 7, 7]], device="cuda")
    ca, cb = torch.randn(2, 3, device="cuda"), torch.randn(2, 3, device="cuda")

    def f(h, W):
        r = m.token_logprobs(h, y, W, softcap=5.0, temperature=0.8, top_k=2)
        assert r.top_ids.shape == (2, 3, 2)
        return (r.logp * ca).sum() + (r.entropy * cb).sum()
    f(h, W).backward()
    with torch.no_grad():
        for _ in range(4):
            dh, dw = torch.randn_like(h), torch.randn_like(W)
            n = float((dh.square().sum() + dw.square().sum()).sqrt())
            dh, dw = dh / n * 2.0 ** -7, dw / n * 2.0 ** -7
            num = float(f(h + dh, W + dw) - f(h - dh, W - dw)) * 2.0 ** 6
            ana = float((h.grad * dh).sum() + (W.grad * dw).sum()) * 2.0 ** 7
            assert abs(num - ana) < 1e-2


def test_one_vocabulary_many_chunks_of_tokens():
    """More tokens than one chunk holds: the same bits as the chunks by themselves."""
    import lm_head_linear_amd as m
    N, H, V, K = 8192 + 300, 64, 900, 5
    for dt in (BF, F):
        h, W, y, _, _ = make(N, H, V, dt, ignored=0.0)
        r = m.flce_logprobs(h, W, y, top_k=K)
        one = m.flce_logprobs(h[8192:], W, y[8192:], top_k=K)
        assert all(torch.equal(a[8192:], b) for a, b in zip(r, one))
        y[::3] = IGN
        check_forward(m.flce_logprobs(h, W, y, top_k=K), reference(h, W, y, K, 0.0, 1.0), K, 0.0, 1.0)


@pytest.mark.parametrize("N,dt", [(9, BF), (200, BF), (70, F)])
def test_captured_and_replayed(N, dt):
    import lm_head_linear_amd as m
    H, V, K = 72, 1100, 6
    h, W, y, a, b = make(N, H, V, dt)
    outs = [torch.empty(N, device="cuda") for _ in range(3)]
    tl, ti = torch.empty(N, K, device="cuda"), torch.empty(N, K, dtype=torch.int64, device="cuda")
    dH, dW = torch.empty_like(h), torch.empty_like(W)
    ws = torch.empty(m.flce_logprobs_workspace_size(N, H, V, dt, K), dtype=torch.uint8, device="cuda")
    wb = torch.empty(m.flce_logprobs_backward_workspace_size(N, H, V, dt), dtype=torch.uint8,
                     device="cuda")
    st = torch.empty((), dtype=torch.int32, device="cuda")

    def call():
        m.flce_logprobs(h, W, y, top_k=K, logp=outs[0], entropy=outs[1], lse=outs[2], top_logp=tl,
                        top_ids=ti, workspace=ws, status=st)
        m.flce_logprobs_backward(h, W, y, outs[2], outs[1], a, b, dH=dH, dW=dW, workspace=wb)
    every = [*outs, tl, dH, dW]
    call()
    torch.cuda.synchronize()
    want, ids = [t.clone() for t in every], ti.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for t in every:
            t.fill_(float("nan"))
        ti.fill_(-9), ws.fill_(255), wb.fill_(255)
        torch.randn(512, 512, device="cuda").sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(every, want)) and torch.equal(ti, ids)
