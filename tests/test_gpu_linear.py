"""The linear transform with bias, activation and residual, forward and backward, against
the formulas in float64.

Tolerances, u = 2^-24: a float32 sum of K products is off by a random walk of K roundings
of at most u of the sum of magnitudes S; six standard deviations are 6 sqrt(K) u S (and
K <= 16 counts every rounding: 6 sqrt(K) > K there). An activation's slope is at most 1.13
and its second derivative below 1 in size, so that what z is off by reaches y times 1.13 and
the slope once; forming either takes a dozen roundings of relative size u (16 u of the
larger of 1 and |z|). Stored values are off by half a step, eps / 2. The gradients are
compared with the exact products of the slope that was stored and of dz rounded to its
type (one float32 product and a rounding, which torch does alike), so only the sums' error
and the store's are left."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


def half(dt):
    return torch.finfo(dt).eps / 2


def act64(kind, z):
    f = torch.nn.functional
    return {"none": lambda t: t * 1.0, "relu": torch.relu, "gelu": f.gelu,
            "gelu_tanh": lambda t: f.gelu(t, approximate="tanh"), "silu": f.silu}[kind](z)


def make(N, I, O, dt, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return [t.to(dt).cuda() for t in (r(N, I), 1.5 * r(O, I) / I ** 0.5, 0.3 * r(O), 2 * r(N, O),
                                      r(N, O))]


def inside(got, want, tol, what):
    bad = (got.double() - want).abs() > tol + 1e-37
    assert not bool(bad.any()), (what, int(bad.sum()),
                                 float(((got.double() - want).abs() / tol.clamp_min(1e-37)).max()))


def check(N, I, O, dt, act, bias, residual, ydt=None, seed=0):
    import lm_head_linear_amd as m
    x, w, b, r, dy = make(N, I, O, dt, seed + N + I + O)
    b, r = (b if bias else None), (r if residual else None)
    y, slope = m.flce_linear(x, w, b, r, activation=act, save_slope=True, y_dtype=ydt)
    xd, wd = x.double(), w.double()
    z = xd @ wd.T
    S = xd.abs() @ wd.abs().T
    if bias:
        z, S = z + b.double(), S + b.double().abs()
    ez = 6 * (I + 1) ** 0.5 * U * S
    zz = z.clone().requires_grad_()
    a = act64(act, zz)
    d, = torch.autograd.grad(a.sum(), zz)
    want = a.detach() + (r.double() if residual else 0)
    odt = ydt or dt
    assert y.dtype == odt
    rest = 1.13 * ez + 16 * U * z.abs().clamp_min(1) + (U * r.double().abs() if residual else 0)
    inside(y, want, half(odt) * want.abs() * 1.02 + rest, "y")
    if act == "none":
        assert slope is None
    elif act == "relu":                     # which side of zero only a z near it leaves open
        assert bool(((slope.double() == d) | (z.abs() <= ez)).all())
    else:
        sdt = torch.float16 if dt == torch.bfloat16 else dt
        assert slope.dtype == sdt
        # a half below 2^-14 is a multiple of 2^-24
        inside(slope, d, 2.0 ** -25 + half(sdt) * d.abs() * 1.02 + ez + 16 * U * z.abs().clamp_min(1), "slope")
    dx, dw, db = m.flce_linear_backward(dy, x, w, slope, bias=bias)
    full = dy.float() if slope is None else dy.float() * slope.float()
    dz, fd = full.to(dt).double(), full.double()
    want = dz @ wd
    inside(dx, want, half(dt) * want.abs() * 1.02 + 6 * O ** 0.5 * U * (dz.abs() @ wd.abs()), "dx")
    want = dz.T @ xd
    inside(dw, want, half(dt) * want.abs() * 1.02 + 6 * N ** 0.5 * U * (dz.abs().T @ xd.abs()), "dw")
    if bias:
        want = fd.sum(0)
        inside(db, want, half(dt) * want.abs() * 1.02 + 6 * (N + 4) ** 0.5 * U * fd.abs().sum(0), "db")
    else:
        assert db is None


SIZES = [(1, 1, 1), (1, 64, 64), (3, 5, 7), (2, 4096, 100), (17, 64, 203), (130, 257, 129),
         (64, 40, 4096), (257, 515, 701), (300, 128, 1000), (1000, 63, 65), (515, 1024, 256),
         (16, 1024, 1024), (33, 2000, 77), (48, 777, 1030), (128, 512, 640), (2000, 9, 3)]


@pytest.mark.parametrize("N,I,O", SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_sizes(N, I, O, dt):
    for i, act in enumerate(ACTS):
        check(N, I, O, dt, act, bias=i % 2 == 0, residual=i in (0, 1, 4), seed=i)


@pytest.mark.parametrize("N,I,O", [(1, 64, 32768), (5, 129, 33001), (16, 130, 32770), (33, 256, 40000),
                                   (48, 65, 32769), (100, 40, 33333), (128, 128, 32800)])
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
def test_wide_weights(N, I, O, act):
    check(N, I, O, torch.bfloat16, act, act != "none", act == "none")
    # rows of x apart: another kernel where they are odd, the same sums to their error
    import lm_head_linear_amd as m
    x, w, b, r, _ = make(N, I, O, torch.bfloat16, 4)
    wide = torch.zeros(N, I + 13, device="cuda").bfloat16()
    wide[:, 8:8 + I] = x
    y, _ = m.flce_linear(wide[:, 8:8 + I], w, b, r, activation=act)
    want, _ = m.flce_linear(x, w, b, r, activation=act)
    tol = 6 * I ** 0.5 * U * 2 * 1.13 * (x.double().abs() @ w.double().abs().T + 1)
    inside(y, want.double(), tol + 2 * half(torch.bfloat16) * want.double().abs() * 1.02, "y")


@pytest.mark.parametrize("N,I,O", [(1, 512, 1000), (130, 257, 129), (600, 256, 512), (40, 64, 64)])
def test_float32_out_of_bf16_rows(N, I, O):
    import lm_head_linear_amd as m
    x, w, b, _, _ = make(N, I, O, torch.bfloat16, 5)
    y, _ = m.flce_linear(x, w, b, activation="gelu", y_dtype=torch.float32)
    z = x.double() @ w.double().T + b.double()
    S = x.double().abs() @ w.double().abs().T + b.double().abs()
    inside(y, act64("gelu", z), 8 * I ** 0.5 * U * S + 20 * U * z.abs().clamp_min(1), "y")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,I,O", [(2048, 1024, 1024), (3000, 520, 2056), (4096, 2048, 512)])
def test_many_tiles(N, I, O, dt):
    check(N, I, O, dt, "silu", True, True)


@pytest.mark.parametrize("act", ACTS[1:])
def test_far_arguments(act):
    """Activations far from zero keep their relative accuracy: y over z for z to -12, where
    each activation's factor is still a normal number. The factor's exponent is formed in
    float32: an argument a off by u a changes exp(a) by u a of itself; with a to 80 (z^2 / 2
    of gelu, the cubic of gelu_tanh) and a dozen roundings, 200 u."""
    import lm_head_linear_amd as m
    z = torch.linspace(-12, 12, 4097, device="cuda")[:, None].contiguous()
    one = torch.ones(1, 1, device="cuda")
    y, slope = m.flce_linear(z, one, activation=act, save_slope=True)
    zz = z.double().requires_grad_()
    want = {"relu": lambda t: torch.relu(t),
            "gelu": lambda t: t * torch.special.erfc(-t * 0.5 ** 0.5) / 2,
            "gelu_tanh": lambda t: t * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (t + 0.044715 * t ** 3)),
            "silu": lambda t: t * torch.sigmoid(t)}[act](zz)
    inside(y, want.detach(), 200 * U * want.detach().abs() + 1e-36, "y")
    d, = torch.autograd.grad(want.sum(), zz)
    inside(slope, d, 200 * U * (want.detach().abs() * z.double().abs() + d.abs()) + 8 * U * d.abs() + 1e-36
           + (16 * U * (z.double().abs() < 3)), "slope")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [3, 20, 200])
def test_strides_alignment_in_place(dt, N):
    import lm_head_linear_amd as m
    I, O = 131, 75
    big = torch.randn(N, I + 40, device="cuda").to(dt)
    x = big[:, 3:3 + I]
    w, b = torch.randn(O, I, device="cuda").to(dt), torch.randn(O, device="cuda").to(dt)
    res = torch.randn(N, O + 9, device="cuda").to(dt)
    r = res[:, 5:5 + O]
    want, slope = m.flce_linear(x.contiguous(), w, b, r.contiguous(), activation="gelu", save_slope=True)
    out = torch.full((N, O + 6), 7.0, device="cuda").to(dt)
    y, s2 = m.flce_linear(x, w, b, r, activation="gelu", save_slope=True, y=out[:, 1:1 + O])
    assert torch.equal(y, want) and torch.equal(slope, s2)
    assert bool((out[:, :1] == 7).all()) and bool((out[:, 1 + O:] == 7).all())
    got, _ = m.flce_linear(x, w, b, r, activation="gelu", y=r)
    assert torch.equal(got, want) and got.data_ptr() == r.data_ptr()
    dyb = torch.randn(N, O + 3, device="cuda").to(dt)
    dy = dyb[:, 2:2 + O]
    a = m.flce_linear_backward(dy.contiguous(), x.contiguous(), w, slope)
    dxb = torch.full((N, I + 4), 7.0, device="cuda").to(dt)
    c = m.flce_linear_backward(dy, x, w, slope, dx=dxb[:, 3:3 + I])
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    assert bool((dxb[:, :3] == 7).all()) and bool((dxb[:, 3 + I:] == 7).all())
    # without an activation dz is dy itself, its rows strided
    a = m.flce_linear_backward(dy.contiguous(), x.contiguous(), w)
    c = m.flce_linear_backward(dy, x, w)
    assert all(torch.equal(p, q) for p, q in zip(a, c))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,I,O", [(37, 65, 129), (300, 256, 512)])
def test_accumulate_and_parts(dt, N, I, O):
    import lm_head_linear_amd as m
    x, w, _, _, dy = make(N, I, O, dt, 3)
    slope = torch.rand(N, O, device="cuda").to(torch.float16 if dt == torch.bfloat16 else dt)
    dx, dw, db = m.flce_linear_backward(dy, x, w, slope)
    one = m.flce_linear_backward(dy, x, w, slope, want_dweight=False, bias=False)
    assert torch.equal(one[0], dx) and one[1] is None and one[2] is None
    one = m.flce_linear_backward(dy, x, w, slope, want_dx=False, bias=False)
    assert one[0] is None and torch.equal(one[1], dw)
    one = m.flce_linear_backward(dy, x, w, slope, want_dx=False, want_dweight=False)
    assert one[:2] == (None, None) and torch.equal(one[2], db)
    # added to: one rounding of the float32 sum
    dw0, db0 = torch.randn(O, I, device="cuda").to(dt), torch.randn(O, device="cuda").to(dt)
    _, dw2, db2 = m.flce_linear_backward(dy, x, w, slope, dweight=dw0.clone(), dbias=db0.clone(),
                                         accumulate=True)
    for got, old, new in ((dw2, dw0, dw), (db2, db0, db)):
        want = old.double() + new.double()
        # `new` here was rounded once itself
        inside(got, want, half(dt) * (want.abs() + new.double().abs()) * 1.02
               + U * (old.double().abs() + new.double().abs()), "added")


def test_no_rows():
    import lm_head_linear_amd as m
    for dt in (torch.bfloat16, torch.float32):
        x, w = torch.empty(0, 8, device="cuda", dtype=dt), torch.ones(5, 8, device="cuda", dtype=dt)
        y, s = m.flce_linear(x, w, activation="silu", save_slope=True)
        assert y.shape == (0, 5) and s.shape == (0, 5)
        dx, dw, db = m.flce_linear_backward(y, x, w, s)
        assert dx.shape == (0, 8) and not dw.any() and not db.any()
        dw, db = torch.ones_like(w), torch.ones(5, device="cuda", dtype=dt)
        m.flce_linear_backward(y, x, w, s, dweight=dw, dbias=db, accumulate=True)
        assert bool((dw == 1).all()) and bool((db == 1).all())


def test_nan_and_inf_stay_in_their_rows():
    """Row 1 of x holds NaN, row 2 inf: the other rows are what they are without them."""
    import lm_head_linear_amd as m
    for dt in (torch.bfloat16, torch.float32):
        for N, I, O in ((5, 70, 33), (140, 70, 133), (300, 256, 512)):
            x, w, b, r, dy = make(N, I, O, dt, 9)
            clean, _ = m.flce_linear(x, w, b, r, activation="gelu_tanh")
            x[1, 3], x[2, I - 1] = float("nan"), float("inf")
            y, _ = m.flce_linear(x, w, b, r, activation="gelu_tanh")
            keep = torch.ones(N, dtype=torch.bool)
            keep[1:3] = False
            assert torch.equal(y[keep], clean[keep]) and bool(y[1].isnan().all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", [(5, 40), (2, 3, 40)])
def test_autograd_against_float64_and_differences(act, shape):
    import lm_head_linear_amd as m
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, w, b, res, c = r(*shape), r(24, 40) / 6, r(24), r(*shape[:-1], 24), r(*shape[:-1], 24)
    leaves = [t.requires_grad_() for t in (x, w, b, res)]
    (m.fused_linear(*leaves, activation=act) * c).sum().backward()
    d = [t.detach().double().requires_grad_() for t in leaves]

    def f(p):
        return (act64(act, p[0] @ p[1].T + p[2]) + p[3]) * c.double()
    f(d).sum().backward()
    for got, want in zip(leaves, d):
        assert torch.allclose(got.grad.double(), want.grad, rtol=2e-5, atol=2e-5)
    for i in range(4):                       # a step along the gradient
        p = [t.detach() for t in d]
        h = 1e-6
        up = [q + h * d[i].grad if j == i else q for j, q in enumerate(p)]
        dn = [q - h * d[i].grad if j == i else q for j, q in enumerate(p)]
        slope = float((f(up).sum() - f(dn).sum()) / (2 * h))
        assert abs(slope - float((leaves[i].grad.double() * d[i].grad).sum())) < 1e-4 * abs(slope) + 1e-6


def test_head_transform_in_a_tied_model_and_a_graph():
    """A step of a model with the transform in front of its head: eager, and captured and
    replayed with eager work between."""
    import lm_head_linear_amd as m
    torch.manual_seed(0)
    t = m.TiedLMHead(500, 64, transform="silu", device="cuda", dtype=torch.bfloat16)
    x, y = torch.randint(0, 500, (3, 30), device="cuda"), torch.randint(0, 500, (3, 30), device="cuda")
    mask = m.DropoutMask(0.1, 3)

    def step():
        e = t.embed(x, mask)
        loss = t.loss(torch.tanh(e), y, residual=e, dropout=m.DropoutMask(0.1, 3, 1))
        return [loss.detach(), *torch.autograd.grad(loss, list(t.parameters()))]
    want = [v.clone() for v in step()]
    assert all(bool(torch.isfinite(v.float()).all()) for v in want) and len(want) == 5
    assert bool(t.transform.weight is not None) and all(bool(v.any()) for v in want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))


def test_streams_and_refusals():
    import lm_head_linear_amd as m
    x, w, b, r, dy = make(500, 256, 300, torch.bfloat16, 2)
    want = m.flce_linear(x, w, b, r, activation="silu")[0]
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream() for _ in range(3)]
    for st in streams:
        with torch.cuda.stream(st):
            outs.append(m.flce_linear(x, w, b, r, activation="silu")[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    for bad in (lambda: m.flce_linear(x, w[:, :8], b), lambda: m.flce_linear(x, w.float()),
                lambda: m.flce_linear(x, w, b[:3]), lambda: m.flce_linear(x, w, activation="tanh"),
                lambda: m.flce_linear(x, w, y_dtype=torch.float16),
                lambda: m.flce_linear(x, w, slope=torch.empty_like(r)),
                lambda: m.flce_linear(x.cpu(), w), lambda: m.flce_linear(x.t(), w),
                lambda: m.flce_linear_backward(dy, x, w, accumulate=True),
                lambda: m.flce_linear_backward(dy[:3], x, w),
                lambda: m.fused_linear(x, w, residual=r[:3])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.FlceError):
        m.flce_linear(x, w, residual=r, activation="silu", slope=r.view(torch.float16))
    with pytest.raises(m.FlceError):
        m.flce_linear(x.float(), w.float(), y_dtype=torch.bfloat16)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,I,O", [(7110, 495, 211), (79, 130, 3428), (3000, 64, 64), (5000, 33, 7), (130, 72, 2048)])
def test_split_gradients(dt, N, I, O):
    """Products of few tiles and a long k, cut into segments: both, one of them, added to."""
    import lm_head_linear_amd as m
    check(N, I, O, dt, "silu", True, False)
    x, w, _, _, dy = make(N, I, O, dt, 3)
    a = m.flce_linear_backward(dy, x, w)
    b = m.flce_linear_backward(dy, x, w, want_dx=False, bias=False)
    c = m.flce_linear_backward(dy, x, w, want_dweight=False, bias=False)
    assert torch.equal(a[1], b[1]) and torch.equal(a[0], c[0])
    big = torch.full((N, I + 5), 7.0, device="cuda").to(dt)
    d = m.flce_linear_backward(dy, x, w, dx=big[:, 2:2 + I], dweight=torch.zeros_like(w),
                               dbias=torch.zeros(O, device="cuda", dtype=dt), accumulate=True)
    assert all(torch.equal(p, q) for p, q in zip(a, d))
    assert bool((big[:, :2] == 7).all()) and bool((big[:, 2 + I:] == 7).all())
