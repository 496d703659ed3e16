"""RMS norm with the residual's addition, forward and backward, against the
formulas in float64.

Tolerances: a stored value is off by at most half a step of its type (eps / 2 of
the value); the float32 arithmetic before it adds relative errors of u = 2^-24 a
rounding. A sum over a row goes through chains of at most H / 64 / waves + 10
additions, below 100 at every width here, so a mean is off by 100 u of the sum of
magnitudes and rstd (a square root) by half of that; a dozen roundings follow.
dweight sums N rows in chains of at most N / 1024 + 25, of rows up to 2 KiB (of which a
workgroup takes up to 16 at a time) N / 2048 + 40; both stay below the bound's
N / 1024 + 25 with the 70 for the roundings of each term."""
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


def half(dt):
    return torch.finfo(dt).eps / 2


def make(N, H, dt, seed, wdt=None, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((2 * r(N, H)).to(dt), (4 * r(N, H)).to(dt), (1 - offset + 0.2 * r(H)).to(wdt or dt),
            (0.1 * r(N, H)).to(dt), (0.1 * r(N, H)).to(dt))


def reference(s, w, offset, eps, dy=None, ds=None):
    v, w = s.double().cpu(), w.double().cpu() + offset
    q = 1 / ((v * v).mean(1, keepdim=True) + eps).sqrt()
    n = v * q
    if dy is None:
        return n * w, q[:, 0]
    dy = dy.double().cpu()
    g = dy * w
    dx = q * (g - n * (g * n).mean(1, keepdim=True))
    mag = q * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if ds is not None:
        dx = dx + ds.double().cpu()
        mag = mag + ds.double().cpu().abs()
    return dx, mag, (dy * n).sum(0), (dy * n).abs().sum(0)


def close(got, ref, dt, slack, what):
    got = got.double().cpu()
    tol = half(dt) * ref.abs() * (1 + 2.0 ** -6) + slack + 1e-37
    bad = (got - ref).abs() > tol
    assert not bool(bad.any()), (what, int(bad.sum()), float(((got - ref).abs() / tol).max()))


CASES = [(1, 4096, torch.bfloat16), (16, 4096, torch.bfloat16), (37, 1, torch.float32),
         (5, 2, torch.bfloat16), (300, 513, torch.bfloat16), (2500, 1024, torch.bfloat16),
         (64, 2047, torch.float32), (1030, 515, torch.float32), (9, 8200, torch.bfloat16),
         (7, 16384, torch.float32), (3, 40001, torch.bfloat16), (2, 33000, torch.float32),
         # rows that share a workgroup: 16, 8, 4 and 2 of them, the last one part filled
         (1, 64, torch.bfloat16), (1003, 128, torch.bfloat16), (20011, 100, torch.bfloat16),
         (333, 200, torch.bfloat16), (70, 60, torch.float32), (9001, 121, torch.float32),
         (1001, 250, torch.float32), (517, 511, torch.bfloat16), (45, 1000, torch.bfloat16),
         (4099, 512, torch.float32)]


@pytest.mark.parametrize("N,H,dt", CASES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward_and_backward(N, H, dt, residual):
    import lm_head_linear_amd as m
    offset = 1.0 if residual else 0.0
    x, r, w, dy, ds = (t.cuda() for t in make(N, H, dt, N + H, offset=offset))
    y, s, rstd = m.flce_rms_norm(x, w, r if residual else None, eps=1e-5, weight_offset=offset)
    want_s = (x.float() + r.float()).to(dt) if residual else x
    assert torch.equal(s, want_s)
    ry, rq = reference(s, w, offset, 1e-5)
    close(rstd, rq, torch.float32, 60 * U * rq, "rstd")
    close(y, ry, dt, 70 * U * ry.abs(), "y")
    dx, dw = m.flce_rms_norm_backward(dy, s, w, rstd, ds if residual else None,
                                      weight_offset=offset)
    rx, mag, rw, wmag = reference(s, w, offset, 1e-5, dy, ds if residual else None)
    close(dx, rx, dt, 300 * U * mag, "dx")
    close(dw, rw, dt, (N / 1024 + 25 + 70) * U * wmag, "dw")
    # the same bits again, and dw alone left out
    dx2, dw2 = m.flce_rms_norm_backward(dy, s, w, rstd, ds if residual else None,
                                        weight_offset=offset)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    dx3, none = m.flce_rms_norm_backward(dy, s, w, rstd, ds if residual else None,
                                         weight_offset=offset, want_dweight=False)
    assert none is None and torch.equal(dx, dx3)


def test_float32_weight_with_bf16_rows():
    import lm_head_linear_amd as m
    N, H, dt = 130, 777, torch.bfloat16
    x, r, w, dy, ds = (t.cuda() for t in make(N, H, dt, 5, wdt=torch.float32))
    y, s, rstd = m.flce_rms_norm(x, w, r)
    close(y, reference(s, w, 0.0, 1e-6)[0], dt, 70 * U * 20, "y")
    dx, dw = m.flce_rms_norm_backward(dy, s, w, rstd, ds)
    rx, mag, rw, wmag = reference(s, w, 0.0, 1e-6, dy, ds)
    assert dw.dtype == torch.float32
    close(dx, rx, dt, 300 * U * mag, "dx")
    close(dw, rw, torch.float32, 100 * U * wmag, "dw")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_strides_in_place_and_untouched_neighbours(dt):
    """Rows of a wider buffer at an odd offset, read and written in place: the
    same bits as dense ones, and nothing beside the rows changes."""
    import lm_head_linear_amd as m
    N, H, P = 33, 1027, 1100
    x, r, w, dy, ds = (t.cuda() for t in make(N, H, dt, 9))
    y, s, rstd = m.flce_rms_norm(x, w, r)
    dx, dw = m.flce_rms_norm_backward(dy, s, w, rstd, ds)

    def wide(t):
        b = torch.full((N, P), 7.0, dtype=dt, device="cuda")
        v = b[:, 3:3 + H]
        v.copy_(t)
        return b, v
    bx, vx = wide(x)
    br, vr = wide(r)
    y2, s2, q2 = m.flce_rms_norm(vx, w, vr, y=vx, s=vr)
    assert y2.data_ptr() == vx.data_ptr() and s2.data_ptr() == vr.data_ptr()
    assert torch.equal(vx, y) and torch.equal(vr, s) and torch.equal(q2, rstd)
    by, vy = wide(dy)
    bd, vd = wide(ds)
    acc = dw.clone()
    dx2, dw2 = m.flce_rms_norm_backward(vy, vr, w, rstd, vd, dx=vy, dweight=acc,
                                        accumulate_dweight=True)
    assert torch.equal(vy, dx)
    close(dw2, 2 * dw.double().cpu(), dt, 1e-6 * dw.double().cpu().abs() + half(dt) * dw.double().cpu().abs(), "dw")
    for b in (bx, br, by, bd):
        assert bool((b[:, :3] == 7).all()) and bool((b[:, 3 + H:] == 7).all())


def test_no_rows_zero_rows_and_not_finite():
    import lm_head_linear_amd as m
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, s, rstd = m.flce_rms_norm(e, w, e)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dw = torch.full((64,), 3.0, dtype=torch.bfloat16, device="cuda")
    m.flce_rms_norm_backward(e, e, w, rstd, dweight=dw, accumulate_dweight=True)
    assert bool((dw == 3).all())
    m.flce_rms_norm_backward(e, e, w, rstd, dweight=dw)
    assert bool((dw == 0).all())
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 5] = float("inf")
    x[2, 5] = float("nan")
    y, _, rstd = m.flce_rms_norm(x, w)
    assert bool((y[0] == 0).all()) and float(rstd[0]) == pytest.approx(1e3, rel=1e-6)
    assert float(rstd[1]) == 0 and bool(y[1, 5].isnan()) and bool((y[1, 6:] == 0).all())
    assert bool(y[2].isnan().all())


def test_gradients_against_differences():
    """The autograd form against central differences of its own forward, in
    float32: a step of 2^-6 leaves a truncation error of order 2^-12 and a
    rounding error of a few u / 2^-6 of a sum of 30 terms."""
    import lm_head_linear_amd as m
    torch.manual_seed(3)
    x = torch.randn(2, 3, 5, device="cuda", requires_grad=True)
    r = torch.randn(2, 3, 5, device="cuda", requires_grad=True)
    w = (1 + 0.1 * torch.randn(5, device="cuda")).requires_grad_()
    cy, cs = torch.randn(2, 3, 5, device="cuda"), torch.randn(2, 3, 5, device="cuda")

    def f(x, r, w):
        y, s = m.fused_rms_norm(x, w, r, eps=1e-3)
        return (y * cy).sum() + (s * cs).sum()
    f(x, r, w).backward()
    assert x.grad.data_ptr() != r.grad.data_ptr()
    with torch.no_grad():
        for t in (x, r, w):
            for i in range(t.numel()):
                d = torch.zeros_like(t)
                d.view(-1)[i] = 2.0 ** -6
                args = [(a + d, a - d) if a is t else (a, a) for a in (x, r, w)]
                num = (f(*[a[0] for a in args]) - f(*[a[1] for a in args])) * 2.0 ** 5
                assert abs(float(num) - float(t.grad.view(-1)[i])) < 5e-3


def test_captured_and_replayed():
    import lm_head_linear_amd as m
    N, H, dt = 260, 1024, torch.bfloat16
    x, r, w, dy, ds = (t.cuda() for t in make(N, H, dt, 77))
    y, s, dx = (torch.empty(N, H, dtype=dt, device="cuda") for _ in range(3))
    q, dw = torch.empty(N, device="cuda"), torch.empty(H, dtype=dt, device="cuda")
    ws = torch.empty(m.flce_rms_norm_backward_workspace_size(N, H), dtype=torch.uint8, device="cuda")

    def call():
        m.flce_rms_norm(x, w, r, y=y, s=s, rstd=q)
        m.flce_rms_norm_backward(dy, s, w, q, ds, dx=dx, dweight=dw, workspace=ws)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, s, q, dx, dw)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for t in (y, s, q, dx, dw):
            t.fill_(float("nan"))
        torch.randn(512, 512, device="cuda").sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, s, q, dx, dw), want))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_any_layout_through_autograd(dt):
    """Transposed, sliced and broadcast rows give the bits of their copies, and a
    broadcast input's gradient is the sum over its copies."""
    import lm_head_linear_amd as m
    x, r, w, dy, ds = (t.cuda() for t in make(12, 40, dt, 11))
    want, s, _ = m.flce_rms_norm(x, w, r)
    layouts = [x.t().contiguous().t(), torch.stack([x, x], 2)[:, :, 0], x.view(3, 4, 40)]
    for a in layouts:
        y, t = m.fused_rms_norm(a, w, r.view(a.shape))
        assert torch.equal(y.reshape(12, 40), want) and torch.equal(t.reshape(12, 40), s)
    one = x[:1].clone().requires_grad_()
    y = m.fused_rms_norm(one.expand(12, 40), w)
    assert torch.equal(y, m.flce_rms_norm(one.detach().expand(12, 40).contiguous(), w)[0])
    y.backward(dy)
    rows, _ = m.flce_rms_norm_backward(dy, one.detach().expand(12, 40).contiguous(), w,
                                       m.flce_rms_norm(one.detach(), w)[2].expand(12).contiguous())
    assert torch.equal(one.grad, rows.sum(0, keepdim=True))


def test_a_second_derivative_and_a_foreign_workspace_are_refused():
    import lm_head_linear_amd as m
    x, r, w, dy, ds = (t.cuda() for t in make(4, 24, torch.float32, 12))
    x.requires_grad_()
    (g,) = torch.autograd.grad(m.fused_rms_norm(x, w).square().sum(), x,
                               create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
    y, s, q = m.flce_rms_norm(x.detach(), w)
    need = m.flce_rms_norm_backward_workspace_size(4, 24)
    with pytest.raises(ValueError, match="workspace"):
        m.flce_rms_norm_backward(dy, s, w, q, workspace=torch.empty(need, dtype=torch.uint8))
