"""Embedding lookup with scaling and its gradient by sorted tokens.

The lookup is exact: one float32 product, rounded once. A gradient row of n
tokens is a float32 sum of n values (n roundings of u = 2^-24 of the magnitudes'
sum), scaled (one more, one more when added to an existing row) and rounded to
half a step of its type."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


def ids(N, V, law, g):
    if law == "uniform":
        t = torch.randint(0, V, (N,), generator=g)
    elif law == "same":
        t = torch.full((N,), V // 2)
    elif law == "runs":                    # ids whose runs end at every offset of a window
        t = torch.repeat_interleave(torch.arange(N), 1 + torch.arange(N) % 67)[:N] % V
        t = t[torch.randperm(N, generator=g)]
    else:                                  # few very frequent ids
        t = (V * torch.rand(N, generator=g) ** 6).long().clamp(0, V - 1)
    return t


def make(N, H, V, dt, law, seed=1):
    g = torch.Generator().manual_seed(seed)
    t = ids(N, V, law, g)
    pad = -7
    if N > 3:
        t[torch.randperm(N, generator=g)[: N // 10 + 1]] = pad
    W = torch.randn(V, H, generator=g).to(dt)
    d = (0.1 * torch.randn(N, H, generator=g)).to(dt)
    return t.cuda(), W.cuda(), d.cuda(), pad


def check_grad(got, tokens, dout, scale, gdt, base=None):
    V = got.shape[0]
    live = (tokens >= 0) & (tokens < V)
    t, d = tokens[live], dout[live].double()
    ref = torch.zeros(V, d.shape[1], dtype=torch.float64, device="cuda").index_add_(0, t, d) * scale
    mag = torch.zeros_like(ref).index_add_(0, t, d.abs()) * abs(scale)
    n = torch.bincount(t, minlength=V).double()[:, None]
    if base is not None:
        ref += base.double()
        mag += base.double().abs()
    err = (got.double() - ref).abs()
    tol = torch.finfo(gdt).eps / 2 * ref.abs() * (1 + 2.0 ** -6) + (n + 3) * U * mag
    assert not bool((err > tol).any()), float((err - tol).max())


CASES = [(1, 8, 1, torch.bfloat16, "uniform"), (3, 1, 5, torch.float32, "uniform"),
         (31, 513, 40, torch.bfloat16, "uniform"), (33, 100, 7, torch.float32, "same"),
         (1000, 1024, 600, torch.bfloat16, "zipf"), (4096, 131, 1000, torch.bfloat16, "runs"),
         (4097, 520, 70000, torch.float32, "zipf"), (16384, 264, 300, torch.bfloat16, "runs"),
         (16385, 136, 70001, torch.bfloat16, "zipf"), (50000, 72, 257, torch.float32, "zipf"),
         (32768, 40, 9000, torch.bfloat16, "runs"), (1024, 65, 300, torch.float32, "runs"),
         (32769, 40, 9000, torch.float32, "zipf"),
         (40000, 64, 3, torch.bfloat16, "same")]


@pytest.mark.parametrize("N,H,V,dt,law", CASES)
def test_lookup_and_gradient(N, H, V, dt, law):
    import lm_head_linear_amd as m
    tokens, W, dout, pad = make(N, H, V, dt, law)
    scale = 1.7
    out = m.flce_embedding(tokens, W, scale=scale, padding_index=pad)
    want = (W[tokens.clamp_min(0)].float() * torch.tensor(scale, dtype=torch.float32, device="cuda")).to(dt)
    want[tokens == pad] = 0
    assert torch.equal(out, want)
    dW = m.flce_embedding_backward(tokens, dout, V, scale=scale, padding_index=pad)
    check_grad(dW, tokens, dout, scale, dt)
    again = m.flce_embedding_backward(tokens, dout, V, scale=scale, padding_index=pad)
    assert torch.equal(dW, again)
    # added to what is there: rows without tokens keep their bits
    base = torch.randn(V, H, device="cuda").to(dt)
    acc = base.clone()
    m.flce_embedding_backward(tokens, dout, V, scale=scale, padding_index=pad, dW=acc,
                              accumulate_dW=True)
    check_grad(acc, tokens, dout, scale, dt, base)
    hit = torch.zeros(V, dtype=torch.bool, device="cuda")
    hit[tokens[tokens != pad]] = True
    assert torch.equal(acc[~hit], base[~hit])


def test_float32_gradient_of_bf16_rows():
    import lm_head_linear_amd as m
    tokens, W, dout, pad = make(3000, 200, 500, torch.bfloat16, "zipf")
    dW = m.flce_embedding_backward(tokens, dout, 500, padding_index=pad, grad_dtype=torch.float32)
    assert dW.dtype == torch.float32
    check_grad(dW, tokens, dout, 1.0, torch.float32)


@pytest.mark.parametrize("N", [200, 20000])
def test_bad_ids_and_padding_inside_the_table(N):
    import lm_head_linear_amd as m
    V, H = 100, 72
    tokens, W, dout, _ = make(N, H, V, torch.bfloat16, "uniform")
    tokens = tokens.clamp_min(0)
    st = torch.full((), -1, dtype=torch.int32, device="cuda")
    out = m.flce_embedding(tokens, W, padding_index=5, status=st)
    assert int(st) == 0 and bool((out[tokens == 5] == 0).all())
    dW = m.flce_embedding_backward(tokens, dout, V, padding_index=5, status=st)
    assert int(st) == 0 and bool((dW[5] == 0).all())
    bad = tokens.clone()
    bad[[3, 50]] = torch.tensor([V, -2], device="cuda")
    bad[60] = 2 ** 40
    out = m.flce_embedding(bad, W, padding_index=5, status=st)
    assert int(st) == 5
    rows = out.isnan().all(1)
    assert bool(rows[[3, 50, 60]].all()) and int(out.isnan().any(1).sum()) == 3
    st.fill_(-1)
    dW = m.flce_embedding_backward(bad, dout, V, padding_index=5, status=st)
    assert int(st) == 5
    check_grad(dW, torch.where(bad == 5, -1, bad), dout, 1.0, torch.bfloat16)


def test_all_padding_and_no_tokens():
    import lm_head_linear_amd as m
    W = torch.randn(9, 40, device="cuda")
    for n in (0, 70):
        t = torch.full((n,), -100, device="cuda")
        assert bool((m.flce_embedding(t, W) == 0).all())
        d = torch.randn(n, 40, device="cuda")
        dW = torch.full((9, 40), 2.0, device="cuda")
        m.flce_embedding_backward(t, d, 9, dW=dW, accumulate_dW=True)
        assert bool((dW == 2).all())
        m.flce_embedding_backward(t, d, 9, dW=dW)
        assert bool((dW == 0).all())


def test_strided_rows():
    import lm_head_linear_amd as m
    N, H, V = 90, 130, 50
    tokens, W, dout, pad = make(N, H, V, torch.bfloat16, "zipf")
    buf = torch.full((N, 200), 3.0, dtype=torch.bfloat16, device="cuda")
    m.flce_embedding(tokens, W, padding_index=pad, out=buf[:, 5:135])
    assert torch.equal(buf[:, 5:135], m.flce_embedding(tokens, W, padding_index=pad))
    assert bool((buf[:, :5] == 3).all()) and bool((buf[:, 135:] == 3).all())
    buf[:, 5:135] = dout
    assert torch.equal(m.flce_embedding_backward(tokens, buf[:, 5:135], V, padding_index=pad),
                       m.flce_embedding_backward(tokens, dout, V, padding_index=pad))


def test_autograd_matches_the_dense_product():
    import lm_head_linear_amd as m
    V, H = 30, 24
    W = torch.randn(V, H, device="cuda", requires_grad=True)
    t = torch.randint(0, V, (4, 7), device="cuda")
    c = torch.randn(4, 7, H, device="cuda")
    (m.fused_embedding(t, W, scale=2.0) * c).sum().backward()
    W2 = W.detach().double().requires_grad_()
    ((W2[t] * 2.0) * c.double()).sum().backward()
    # at most 28 terms a row: 30 roundings of their magnitudes, below 10 each
    assert float((W.grad.double() - W2.grad).abs().max()) < 30 * U * 28 * 10


def test_captured_and_replayed():
    import lm_head_linear_amd as m
    N, H, V = 20000, 96, 3000
    tokens, W, dout, pad = make(N, H, V, torch.bfloat16, "zipf")
    out, dW = torch.empty(N, H, dtype=W.dtype, device="cuda"), torch.empty_like(W)
    ws = torch.empty(m.flce_embedding_backward_workspace_size(N, H, V), dtype=torch.uint8,
                     device="cuda")
    st = torch.empty((), dtype=torch.int32, device="cuda")

    def call():
        m.flce_embedding(tokens, W, padding_index=pad, out=out, status=st)
        m.flce_embedding_backward(tokens, dout, V, padding_index=pad, dW=dW, workspace=ws)
    call()
    torch.cuda.synchronize()
    want = out.clone(), dW.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.fill_(float("nan")), dW.fill_(float("nan")), ws.fill_(255)
        torch.randn(512, 512, device="cuda").sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(dW, want[1]) and int(st) == 0
