"""Dropout, the linear transform and sampling where an element's offset passes 32 bits, and at
the ends of what their checks allow: rows around 2^31 and 2^32 elements and the last ones
against the formulas, tolerances of their own tests."""
import math

import pytest
import torch

from tests import test_gpu_dropout as td
from tests import test_gpu_linear as tl
from tests import test_gpu_sample as ts

pytestmark = pytest.mark.gpu
U, BF, F32 = 2.0 ** -24, torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def parts(N, H):
    """Slices of rows at the start, around the elements 2^31 and 2^32, and the last."""
    out = [slice(0, 3)]
    for at in (1 << 31, 1 << 32):
        if at // H + 2 <= N:
            out.append(slice(at // H - 2, at // H + 2))
    return out + [slice(N - 3, N)]


def filled(N, H, seed):
    """bf16 rows of many values without the time that so many normal ones take."""
    t = torch.empty(N, H, device="cuda", dtype=BF)
    g = torch.Generator(device="cuda").manual_seed(seed)
    t[:] = torch.randn(1, H, generator=g, device="cuda").to(BF)
    return t.mul_((0.5 + torch.rand(N, 1, generator=g, device="cuda")).to(BF))


def test_dropout():
    import lm_head_linear_amd as m
    N, H = 65600, 65536
    x, r = filled(N, H, 1), filled(N, H, 2)
    kw = dict(p=0.3, seed=5, offset=9)
    out = m.flce_dropout(x, r, **kw)
    alone = m.flce_dropout(x, **kw)
    for rows in parts(N, H):
        keep, scale = td.keep_mask(rows.stop - rows.start, H, 0.3, 5, 9, row0=rows.start)
        want = torch.where(keep, x[rows].double().cpu() * scale, 0.0)
        td.close(alone[rows], want, BF, 2 * U * want.abs(), "out")
        both = want + r[rows].double().cpu()
        td.close(out[rows], both, BF, 3 * U * (want.abs() + r[rows].double().cpu().abs()), "with residual")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N,H", [(3, (1 << 24) - 1), (2, 1 << 24)])
def test_dropout_of_the_widest_rows(N, H, dt):
    import lm_head_linear_amd as m
    x = torch.ones(N, H, device="cuda", dtype=dt)
    out = m.flce_dropout(x, p=0.5, seed=3)
    for c in (slice(0, 64), slice(H - 70, H)):
        keep, scale = td.keep_mask(N, H, 0.5, 3, 0) if c.start == 0 else (keep, scale)
        assert torch.equal(out[:, c].double().cpu(), keep[:, c].double() * scale)


@pytest.mark.parametrize("N,H", [(1048700, 4096), ((1 << 21) + 37, 24)])
def test_dropout_with_the_norm(N, H):
    """The second size: more rows than one launch of the forward takes, whose mask goes on."""
    import lm_head_linear_amd as m
    x, r, dy = filled(N, H, 1), filled(N, H, 2), filled(N, H, 3)
    w = (1 + 0.2 * torch.randn(H, device="cuda")).to(BF)
    kw = dict(p=0.2, seed=99, offset=7)
    y, s, rstd = m.flce_dropout_norm(x, w, r, eps=1e-5, **kw)
    dx, dres, dw = m.flce_dropout_norm_backward(dy, s, w, rstd, **kw)
    assert bool(torch.isfinite(dw.float()).all())
    edge = 1 << 21
    for rows in parts(N, H) + ([slice(edge - 3, edge + 3)] if N > edge else []):
        keep, scale = td.keep_mask(rows.stop - rows.start, H, 0.2, 99, 7, row0=rows.start)
        drop = torch.where(keep, x[rows].double().cpu() * scale, 0.0)
        td.close(s[rows], drop + r[rows].double().cpu(), BF, 3 * U * (drop.abs() + r[rows].double().cpu().abs()), "s")
        y1, _, q1 = m.flce_rms_norm(s[rows], w, eps=1e-5)
        assert torch.equal(y[rows], y1) and torch.equal(rstd[rows], q1)
        dres1, _ = m.flce_rms_norm_backward(dy[rows], s[rows], w, q1)
        assert torch.equal(dres[rows], dres1)
        d = dres1.double().cpu()
        td.close(dx[rows], torch.where(keep, d * scale, 0.0), BF, (td.half(BF) * scale * 1.02) * d.abs(), "dx")


@pytest.mark.parametrize("O", [32768, 32767])
def test_linear(O):
    """The head's tiles; and rows of an odd length, by way of registers."""
    import lm_head_linear_amd as m
    N, I = 131200, 64
    g = torch.Generator(device="cuda").manual_seed(O)
    x, w, b = (torch.randn(*s, generator=g, device="cuda").to(BF) for s in ((N, I), (O, I), (O,)))
    w /= 8
    r, dy = filled(N, O, 2), filled(N, O, 3)
    y, slope = m.flce_linear(x, w, b, r, activation="silu", save_slope=True)
    dx, dw, db = m.flce_linear_backward(dy, x, w, slope)
    wd = w.double()
    for rows in parts(N, O):
        xd, rd = x[rows].double(), r[rows].double()
        z = xd @ wd.T + b.double()
        S = xd.abs() @ wd.abs().T + b.double().abs()
        ez = 6 * (I + 1) ** 0.5 * U * S
        q = torch.sigmoid(z)
        want = z * q + rd
        tl.inside(y[rows], want, tl.half(BF) * want.abs() * 1.02 + 1.13 * ez
                  + 16 * U * z.abs().clamp_min(1) + U * rd.abs(), "y")
        d = q * (1 + z * (1 - q))
        tl.inside(slope[rows], d, 2.0 ** -25 + 2.0 ** -11 * d.abs() * 1.02 + ez
                  + 16 * U * z.abs().clamp_min(1), "slope")
        dz = (dy[rows].float() * slope[rows].float()).to(BF).double()
        want = dz @ wd
        tl.inside(dx[rows], want, tl.half(BF) * want.abs() * 1.02 + 6 * O ** 0.5 * U * (dz.abs() @ wd.abs()), "dx")
    for cols in (slice(0, 5), slice(O - 5, O)):
        full = dy[:, cols].float() * slope[:, cols].float()
        dz, xd = full.to(BF).double(), x.double()
        want = dz.T @ xd
        tl.inside(dw[cols], want, tl.half(BF) * want.abs() * 1.02 + 6 * N ** 0.5 * U * (dz.abs().T @ xd.abs()), "dw")
        want = full.double().sum(0)
        tl.inside(db[cols], want, tl.half(BF) * want.abs() * 1.02 + 6 * (N + 4) ** 0.5 * U * full.double().abs().sum(0), "db")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N,I,O", [(1, 8, 1 << 24), (2, (1 << 24) - 5, 3), (1 << 22, 8, 8), ((1 << 22) + 1, 3, 5)])
def test_linear_of_one_long_side(N, I, O, dt):
    tl.check(N, I, O, dt, "silu", True, True)


def test_sampling():
    import lm_head_linear_amd as m
    N, V = 33000, 131072
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(N, V, generator=g, device="cuda", dtype=BF).mul_(2)
    u = torch.rand(N, generator=g, device="cuda")
    for kw in (dict(top_k=50, top_p=0.9), dict(top_p=0.9), dict(), dict(temperature=0.0)):
        r = m.flce_sample_logits(z, u, **kw)
        for rows in parts(N, V):
            p = m.flce_sample_logits(z[rows], u[rows], **kw)
            assert torch.equal(p.tokens, r.tokens[rows]) and torch.equal(p.logp, r.logp[rows])


@pytest.mark.parametrize("V,dt", [(1 << 24, F32), ((1 << 24) - 3, BF)])
def test_sampling_from_the_longest_rows(V, dt):
    g = torch.Generator().manual_seed(V)
    z = (2.5 * torch.randn(1, V, generator=g)).to(dt).cuda()
    u = torch.tensor([0.37], device="cuda")
    for kw in (dict(T=0.7, k=50, p=0.9), dict(T=0.8, p=0.9), dict(T=1.0)):
        ts.compare(ts.run(z, u, **kw), z, u, **kw)
    r = ts.run(z, u, T=0.0)
    assert int(r.tokens) == int((z[0] == z[0].max()).nonzero()[0]) and float(r.logp) == 0.0
    z[0, 5] = math.nan
    r = ts.run(z, u, p=0.9)
    assert int(r.tokens) == -1 and math.isnan(float(r.logp))
