"""Dropout from the counter-based generator, alone, with the residual and with the norm,
forward and backward, against the formulas in float64 and a generator in numpy.

Tolerances: a stored value is off by at most half a step of its type (eps / 2 of the
value). Before it stands one float32 product and sum (fused: one rounding, u = 2^-24 of
the sum of magnitudes) with a scale that is itself rounded to float32 (u). With the norm,
s is exact to its rounding and the norm of the s that was stored, so its tolerances are
those of the norm alone: a mean off by 100 u of the sum of magnitudes, a dozen roundings."""
import numpy as np
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


def philox(c, k):
    """Ten rounds of Philox 4x32 on arrays of 32-bit words (uint64 arithmetic)."""
    c, k = [np.uint64(v) if np.isscalar(v) else v.astype(np.uint64) for v in c], list(k)
    m = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & m,
             (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(N, H, p, seed, offset, row0=0):
    nb = (H + 7) // 8
    col, row = np.meshgrid(np.arange(nb), np.arange(row0, row0 + N))
    offset %= 1 << 64
    z = np.zeros_like(col)
    w = philox([col, row, z + (offset & 0xFFFFFFFF), z + (offset >> 32)],
               (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], -1)
    t = min(int(np.floor(p * 65536 + 0.5)), 65535)
    keep = halves.reshape(N, nb * 8)[:, :H] >= t
    return torch.from_numpy(keep), 65536 / (65536 - t)


def half(dt):
    return torch.finfo(dt).eps / 2


def close(got, ref, dt, slack, what):
    got = got.double().cpu()
    tol = half(dt) * ref.abs() * (1 + 2.0 ** -6) + slack + 1e-37
    bad = (got - ref).abs() > tol
    assert not bool(bad.any()), (what, int(bad.sum()), float(((got - ref).abs() / tol).max()))


def make(N, H, dt, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((2 * r(N, H)).to(dt), (4 * r(N, H)).to(dt), (1 + 0.2 * r(H)).to(dt),
            (0.1 * r(N, H)).to(dt), (0.1 * r(N, H)).to(dt))


def test_the_oracles_generator():
    """Published known answers of the generator (Random123's test vectors)."""
    f = 0xFFFFFFFF
    for c, k, want in [((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
                       ((f, f, f, f), (f, f), (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
                       ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
                        (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))]:
        assert tuple(int(v) for v in philox([np.array([x]) for x in c], k)) == want


CASES = [(1, 1, torch.float32), (1, 4096, torch.bfloat16), (37, 1, torch.bfloat16),
         (5, 3, torch.float32), (300, 513, torch.bfloat16), (64, 2047, torch.float32),
         (1030, 515, torch.float32), (9, 8200, torch.bfloat16), (20011, 100, torch.bfloat16),
         (7, 16384, torch.float32), (3, 40001, torch.bfloat16), (2, 33000, torch.float32),
         # more than 2^20 blocks of eight columns: four a thread
         (8200, 1030, torch.bfloat16), (70001, 120, torch.float32)]


@pytest.mark.parametrize("N,H,dt", CASES)
@pytest.mark.parametrize("p", [0.1, 0.0, 0.73])
def test_forward_and_backward(N, H, dt, p):
    import lm_head_linear_amd as m
    x, r, _, dy, _ = (t.cuda() for t in make(N, H, dt, N + H))
    kw = dict(p=p, seed=(N << 33) + 17, offset=(1 << 40) + H)
    keep, scale = keep_mask(N, H, p, kw["seed"], kw["offset"])
    dropped = torch.where(keep, x.double().cpu() * scale, 0.0)
    close(m.flce_dropout(x, **kw), dropped, dt, 2 * U * dropped.abs(), "out")
    want = dropped + r.double().cpu()
    mag = dropped.abs() + r.double().cpu().abs()
    close(m.flce_dropout(x, r, **kw), want, dt, 3 * U * mag, "out with residual")
    dx = torch.where(keep, dy.double().cpu() * scale, 0.0)
    close(m.flce_dropout_backward(dy, **kw), dx, dt, 2 * U * dx.abs(), "dx")


@pytest.mark.parametrize("N,H,dt", [c for c in CASES if c[0] < 8000])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("wide", [False, True])
def test_with_the_norm(N, H, dt, residual, wide):
    """wide: float32 weights with bf16 rows."""
    import lm_head_linear_amd as m
    x, r, w, dy, ds = (t.cuda() for t in make(N, H, dt, N + H))
    if wide:
        w = w.float()
    kw = dict(p=0.2, seed=99, offset=H)
    keep, scale = keep_mask(N, H, 0.2, 99, H)
    y, s, rstd = m.flce_dropout_norm(x, w, r if residual else None, eps=1e-5, weight_offset=0.5,
                                     **kw)
    want = torch.where(keep, x.double().cpu() * scale, 0.0)
    mag = want.abs()
    if residual:
        want, mag = want + r.double().cpu(), mag + r.double().cpu().abs()
    close(s, want, dt, 3 * U * mag, "s")
    # the norm of the s that was stored: the same bits as the norm alone
    y1, _, rstd1 = m.flce_rms_norm(s, w, eps=1e-5, weight_offset=0.5)
    assert torch.equal(y, y1) and torch.equal(rstd, rstd1)
    dx, dres, dw = m.flce_dropout_norm_backward(dy, s, w, rstd, ds, weight_offset=0.5, **kw)
    dres1, dw1 = m.flce_rms_norm_backward(dy, s, w, rstd, ds, weight_offset=0.5)
    assert torch.equal(dres, dres1) and torch.equal(dw, dw1)
    # dx is rounded once, not from the rounded dres: two halves of a step apart at most
    d = dres.double().cpu()
    close(dx, torch.where(keep, d * scale, 0.0), dt, (half(dt) * scale * 1.02) * d.abs(), "dx")
    assert torch.equal(dx.cpu()[~keep], torch.zeros_like(dx.cpu()[~keep]))
    only_x, none, _ = m.flce_dropout_norm_backward(dy, s, w, rstd, ds, weight_offset=0.5,
                                                   want_dresidual=False, want_dweight=False, **kw)
    assert none is None and torch.equal(only_x, dx)


def test_dropped_values_count_as_zero():
    import lm_head_linear_amd as m
    keep, scale = keep_mask(40, 100, 0.5, 5, 0)
    x = torch.ones(40, 100)
    x[~keep] = float("nan")
    x[0, ~keep[0]] = float("inf")
    for dt in (torch.float32, torch.bfloat16):
        out = m.flce_dropout(x.to(dt).cuda(), p=0.5, seed=5)
        assert torch.equal(out.float().cpu(), keep.float() * scale)
        y, s, _ = m.flce_dropout_norm(x.to(dt).cuda(), torch.ones(100, dtype=dt).cuda(), p=0.5, seed=5)
        assert torch.equal(s.float().cpu(), keep.float() * scale)
        assert torch.isfinite(y.float()).all()


def test_masks_rate_and_independence():
    """4e6 values at p = 0.3: the kept share is off by less than 6 standard deviations, and
    two masks agree as often as independent ones (6 standard deviations)."""
    import lm_head_linear_amd as m
    n, p = 2000 * 2048, 0.3
    x = torch.ones(2000, 2048, device="cuda")
    t = int(0.3 * 65536 + 0.5) / 65536
    masks = [m.flce_dropout(x, p=p, seed=s, offset=o) != 0 for s, o in ((1, 0), (1, 1), (2, 0), (1 << 32, 0))]
    for k in masks:
        assert abs(float(k.double().mean()) - (1 - t)) < 6 * (t * (1 - t) / n) ** 0.5
    q = t * t + (1 - t) ** 2
    for i in range(len(masks)):
        for j in range(i):
            same = float((masks[i] == masks[j]).double().mean())
            assert abs(same - q) < 6 * (q * (1 - q) / n) ** 0.5
    # neighbours in a row and in a column
    for a, b in ((masks[0][:, 1:], masks[0][:, :-1]), (masks[0][1:], masks[0][:-1])):
        assert abs(float((a == b).double().mean()) - q) < 6 * (q * (1 - q) / a.numel()) ** 0.5


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_strides_alignment_and_in_place(dt):
    import lm_head_linear_amd as m
    N, H = 77, 203
    big = torch.randn(N, H + 60, device="cuda").to(dt)
    res = torch.randn(N, 2 * H + 9, device="cuda").to(dt)
    x, r = big[:, 7:7 + H], res[:, 3:3 + H]
    kw = dict(p=0.4, seed=7, offset=3)
    want = m.flce_dropout(x.contiguous(), r.contiguous(), **kw)
    out = torch.full((N, H + 31), 7.0, device="cuda").to(dt)
    assert torch.equal(m.flce_dropout(x, r, out=out[:, 5:5 + H], **kw), want)
    assert torch.equal(out[:, :5], torch.full_like(out[:, :5], 7)) and bool((out[:, 5 + H:] == 7).all())
    for inplace in (x, r):
        a, b = big.clone(), res.clone()
        xa, ra = a[:, 7:7 + H], b[:, 3:3 + H]
        assert torch.equal(m.flce_dropout(xa, ra, out=xa if inplace is x else ra, **kw), want)
    w = torch.ones(H, device="cuda").to(dt)
    y, s, _ = m.flce_dropout_norm(x.contiguous(), w, r.contiguous(), **kw)
    b = res.clone()
    y2, s2, _ = m.flce_dropout_norm(x, w, b[:, 3:3 + H], s=b[:, 3:3 + H], **kw)
    assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(s, want)


def test_step_on_the_device_and_wrap():
    import lm_head_linear_amd as m
    x = torch.randn(33, 100, device="cuda")
    step = torch.tensor(5, device="cuda")
    a = m.flce_dropout(x, p=0.5, seed=3, offset=10, step=step)
    assert torch.equal(a, m.flce_dropout(x, p=0.5, seed=3, offset=15))
    step.fill_(-1)
    assert torch.equal(m.flce_dropout(x, p=0.5, seed=3, offset=0, step=step),
                       m.flce_dropout(x, p=0.5, seed=3, offset=(1 << 64) - 1))


def test_captured_with_a_step():
    """Each replay draws the mask of the step it finds, forward and backward alike."""
    import lm_head_linear_amd as m
    x, r = torch.randn(64, 512, device="cuda"), torch.randn(64, 512, device="cuda")
    w, dy = torch.ones(512, device="cuda"), torch.randn(64, 512, device="cuda")
    step = torch.zeros((), dtype=torch.int64, device="cuda")
    kw = dict(p=0.3, seed=11, step=step)

    def work():
        out = m.flce_dropout(x, r, **kw)
        y, s, q = m.flce_dropout_norm(out, w, r, **kw)
        dx, dres, dw = m.flce_dropout_norm_backward(dy, s, w, q, **kw)
        return [out, y, s, dx, dres, dw, m.flce_dropout_backward(dx, **kw)]
    work()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = work()
    seen = []
    for i in range(4):
        step.fill_(i)
        g.replay()
        torch.cuda.synchronize()
        keep = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(keep, work()))
        seen.append(keep[0])
    assert not torch.equal(seen[0], seen[1])


@pytest.mark.parametrize("shape", [(6, 96), (2, 5, 96), (0, 96)])
def test_autograd(shape):
    import lm_head_linear_amd as m
    mask = m.DropoutMask(0.25, 42, 7)
    x = torch.randn(*shape, device="cuda", requires_grad=True)
    r = torch.randn(*shape, device="cuda", requires_grad=True)
    w = torch.rand(96, device="cuda", requires_grad=True)
    n = x.numel() // 96
    keep, scale = keep_mask(n, 96, 0.25, 42, 7) if n else (torch.zeros(0, 96, dtype=torch.bool), 1)
    f = (keep.double() * scale).reshape(shape).cuda()
    c = torch.randn(*shape, device="cuda")
    out = m.fused_dropout(x, mask, r)
    (out * c).sum().backward()
    assert torch.allclose(x.grad, (c * f).float(), rtol=1e-6, atol=0)
    assert torch.equal(r.grad, c)
    x.grad = r.grad = None
    y, s = m.fused_dropout_norm(x, w, mask, r, eps=1e-5)
    ((y * c).sum() + (s * s).sum()).backward()
    xd, rd, wd = (t.detach().double().requires_grad_() for t in (x, r, w))
    sd = xd * f + rd
    yd = sd * torch.rsqrt((sd * sd).mean(-1, keepdim=True) + 1e-5) * wd
    ((yd * c.double()).sum() + (sd * sd).sum()).backward()
    for a, b in ((x, xd), (r, rd), (w, wd)):
        assert torch.allclose(a.grad.double(), b.grad, rtol=1e-4, atol=1e-4)


def test_only_some_gradients_and_a_changed_step():
    import lm_head_linear_amd as m
    x = torch.randn(8, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda")
    y, s = m.fused_dropout_norm(x, w, m.DropoutMask(0.5, 1))
    s.sum().backward()                                   # the sum alone
    keep, scale = keep_mask(8, 64, 0.5, 1, 0)
    assert torch.equal(x.grad.cpu(), keep.float() * scale)
    r = torch.randn(8, 64, device="cuda", requires_grad=True)
    m.fused_dropout(x.detach(), m.DropoutMask(0.5, 1), r).sum().backward()
    assert torch.equal(r.grad, torch.ones_like(r))
    step = torch.zeros((), dtype=torch.int64, device="cuda")
    out = m.fused_dropout(x, m.DropoutMask(0.5, 1, 0, step))
    step += 1
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        out.sum().backward()


def test_two_streams_and_refusals():
    import lm_head_linear_amd as m
    x = torch.randn(4000, 1024, device="cuda")
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            outs.append(m.flce_dropout(x, p=0.5, seed=i))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, m.flce_dropout(x, p=0.5, seed=i))
    for bad in (dict(p=1.0), dict(p=-0.1), dict(p=float("nan")), dict(seed=-1), dict(seed=1 << 64),
                dict(offset=-1), dict(step=torch.zeros(1)), dict(step=torch.zeros(2, dtype=torch.int64,
                                                                                  device="cuda"))):
        with pytest.raises(ValueError):
            m.flce_dropout(x, **{**dict(p=0.5, seed=0), **bad})
    with pytest.raises(ValueError):
        m.flce_dropout(x.half(), p=0.5, seed=0)
    with pytest.raises(ValueError):
        m.flce_dropout(x, x[:, :8], p=0.5, seed=0)
    with pytest.raises(m.FlceError):
        m.flce_dropout(x[:, :512], p=0.5, seed=0, out=x[:, 8:520])
    with pytest.raises(ValueError):
        m.fused_dropout(x, m.DropoutMask(0.5, 0), x[:, :8])
