"""The refusals of dropout, the linear transform and sampling (no GPU): every rule of their
check_args entries, which run the checks of the calls themselves; their workspaces; and the
autograd wrappers with plain torch in the calls' place."""
import os

import pytest
import torch

import lm_head_linear_amd as m
from lm_head_linear_amd import _dropout, _lib, _linear

OK, ARG, UNSUP, WS = _lib.OK, _lib.ERR_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")
M = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__ as g
        g.build()


class Buf:
    """Stands for a device buffer: an address, never read."""

    def __init__(self, at, n=0):
        self.at, self.n = at, n

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def element_size(self):
        return 1


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(residual=None), OK), (dict(N=0, x=None, residual=None, out=None), OK),
    (dict(p=0.0), OK), (dict(p=0.999999), OK), (dict(step=Buf(6 * M)), OK),
    (dict(out=Buf(M)), OK), (dict(out=Buf(2 * M)), OK), (dict(x=Buf(M + 2)), OK),
    (dict(dtype=torch.float32), OK), (dict(seed=(1 << 64) - 1, offset=(1 << 64) - 1), OK),
    (dict(N=-1), ARG), (dict(N=1 << 31), ARG), (dict(H=0), ARG), (dict(H=(1 << 24) + 1), ARG),
    (dict(p=1.0), ARG), (dict(p=-1e-9), ARG), (dict(p=NAN), ARG), (dict(p=INF), ARG),
    (dict(x=None), ARG), (dict(out=None), ARG), (dict(ld_x=23), ARG), (dict(ld_out=0), ARG),
    (dict(ld_res=(1 << 31) + 1), ARG), (dict(out=Buf(M + 2)), ARG), (dict(out=Buf(M), ld_out=25), ARG),
    (dict(out=Buf(2 * M + 48)), ARG), (dict(step=Buf(3 * M)), ARG),
    (dict(x=Buf(M + 1)), UNSUP), (dict(step=Buf(6 * M + 4)), UNSUP),
    (dict(N=(1 << 31) - 1, H=1 << 24, x=Buf(1), residual=None, out=Buf(1 << 62)), UNSUP),
])
def test_dropout(kw, want):
    a = dict(x=Buf(M), residual=Buf(2 * M), N=4, H=24, out=Buf(3 * M))
    a.update(kw)
    assert m.flce_dropout_check_args(**a) == want


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(residual=None), OK), (dict(rstd=None), OK), (dict(y=Buf(M)), OK),
    (dict(s=Buf(M)), OK), (dict(s=Buf(3 * M)), OK), (dict(weight_dtype=torch.float32), OK),
    (dict(N=0, x=None, residual=None, y=None, s=None, rstd=None), OK), (dict(step=Buf(8 * M)), OK),
    (dict(s=None), ARG), (dict(y=None), ARG), (dict(x=None), ARG), (dict(weight=None), ARG),
    (dict(p=1.0), ARG), (dict(p=NAN), ARG), (dict(eps=-1.0), ARG), (dict(weight_offset=INF), ARG),
    (dict(y=Buf(M), s=Buf(M)), ARG), (dict(y=Buf(3 * M)), ARG), (dict(y=Buf(2 * M)), ARG),
    (dict(s=Buf(2 * M)), ARG), (dict(rstd=Buf(5 * M)), ARG), (dict(step=Buf(4 * M)), ARG),
    (dict(step=Buf(6 * M)), ARG), (dict(ld_s=23), ARG), (dict(N=1 << 31), ARG),
    (dict(dtype=torch.float32, weight_dtype=torch.bfloat16), UNSUP), (dict(s=Buf(5 * M + 1)), UNSUP),
])
def test_dropout_norm(kw, want):
    a = dict(x=Buf(M), weight=Buf(2 * M), residual=Buf(3 * M), N=4, H=24, y=Buf(4 * M),
             s=Buf(5 * M), rstd=Buf(6 * M))
    a.update(kw)
    assert m.flce_dropout_norm_check_args(**a) == want


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(ds=None), OK), (dict(dresidual=None), OK),
    (dict(dweight=None, workspace=None), OK), (dict(dx=Buf(M)), OK), (dict(dx=Buf(5 * M)), OK),
    (dict(dresidual=Buf(M), dx=Buf(5 * M)), OK), (dict(dresidual=Buf(5 * M)), OK),
    (dict(dx=Buf(M), dresidual=Buf(M)), ARG), (dict(dx=None), ARG), (dict(dy=None), ARG),
    (dict(s=None), ARG), (dict(rstd=None), ARG), (dict(dx=Buf(2 * M)), ARG), (dict(dx=Buf(M + 2)), ARG),
    (dict(dresidual=Buf(2 * M)), ARG), (dict(dweight=Buf(M)), ARG), (dict(p=1.0), ARG),
    (dict(step=Buf(6 * M)), ARG), (dict(ld_dres=2), ARG), (dict(N=-1), ARG),
    (dict(workspace=Buf(M, 512)), ARG),
    (dict(workspace=None), WS), (dict(workspace=Buf(9 * M, 128)), WS), (dict(workspace=Buf(9 * M + 8, 512)), WS),
])
def test_dropout_norm_backward(kw, want):
    a = dict(dy=Buf(M), s=Buf(2 * M), weight=Buf(3 * M), rstd=Buf(4 * M), ds=Buf(5 * M), N=4, H=24,
             dx=Buf(6 * M), dresidual=Buf(7 * M), dweight=Buf(8 * M), workspace=Buf(9 * M, 512))
    a.update(kw)
    assert m.flce_dropout_norm_backward_check_args(**a) == want


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(bias=None), OK), (dict(residual=None), OK), (dict(slope=None), OK),
    (dict(N=0, x=None, residual=None, y=None, slope=None), OK), (dict(y=Buf(4 * M)), OK),
    (dict(y_dtype=torch.float32), OK), (dict(dtype=torch.float32), OK),
    *[(dict(activation=a), OK) for a in _lib.ACTIVATIONS], (dict(x=Buf(M + 2)), OK),
    (dict(activation=5), ARG), (dict(activation=-1), ARG), (dict(N=-1), ARG), (dict(N=1 << 31), ARG),
    (dict(I=0), ARG), (dict(O=0), ARG), (dict(I=(1 << 24) + 1), ARG), (dict(O=(1 << 24) + 1), ARG),
    (dict(x=None), ARG), (dict(weight=None), ARG), (dict(y=None), ARG), (dict(ld_x=15), ARG),
    (dict(ld_y=23), ARG), (dict(ld_res=23), ARG), (dict(y=Buf(M)), ARG), (dict(y=Buf(2 * M)), ARG),
    (dict(y=Buf(4 * M + 2)), ARG), (dict(y=Buf(4 * M), y_dtype=torch.float32), ARG),
    (dict(slope=Buf(5 * M)), ARG), (dict(slope=Buf(4 * M)), ARG), (dict(slope=Buf(2 * M)), ARG),
    (dict(dtype=torch.float32, y_dtype=torch.bfloat16), UNSUP), (dict(weight=Buf(2 * M + 1)), UNSUP),
])
def test_linear(kw, want):
    a = dict(x=Buf(M), weight=Buf(2 * M), bias=Buf(3 * M), residual=Buf(4 * M), N=4, I=16, O=24,
             activation="silu", y=Buf(5 * M), slope=Buf(6 * M))
    a.update(kw)
    assert m.flce_linear_check_args(**a) == want


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(slope=None), OK), (dict(dx=None, weight=None), OK), (dict(dweight=None, x=None), OK),
    (dict(dbias=None), OK), (dict(dx=None, dweight=None, dbias=None), OK), (dict(accumulate=True), OK),
    (dict(N=0, dy=None, x=None, dx=None), OK), (dict(dtype=torch.float32), OK),
    (dict(dy=None), ARG), (dict(weight=None), ARG), (dict(x=None), ARG), (dict(N=-1), ARG),
    (dict(I=0), ARG), (dict(O=(1 << 24) + 1), ARG), (dict(ld_dy=23), ARG), (dict(ld_x=15), ARG),
    (dict(ld_dx=15), ARG), (dict(dx=Buf(M)), ARG), (dict(dx=Buf(2 * M)), ARG), (dict(dweight=Buf(3 * M)), ARG),
    (dict(dbias=Buf(4 * M)), ARG), (dict(dx=Buf(6 * M)), ARG), (dict(workspace=Buf(M, 1 << 16)), ARG),
    (dict(x=Buf(2 * M + 1)), UNSUP), (dict(workspace=None), WS), (dict(workspace=Buf(8 * M, 100)), WS),
    (dict(workspace=Buf(8 * M + 16, 1 << 16)), WS),
])
def test_linear_backward(kw, want):
    a = dict(dy=Buf(M), x=Buf(2 * M), weight=Buf(3 * M), slope=Buf(4 * M), N=4, I=16, O=24,
             dx=Buf(5 * M), dweight=Buf(6 * M), dbias=Buf(7 * M), workspace=Buf(8 * M, 1 << 16))
    a.update(kw)
    assert m.flce_linear_backward_check_args(**a) == want


SETTINGS = [
    (dict(temperature=0.0), OK), (dict(top_k=5, top_p=0.5, min_p=0.1, softcap=30.0), OK),
    (dict(top_p=1.0, min_p=1.0), OK),
    (dict(temperature=-0.1), ARG), (dict(temperature=NAN), ARG), (dict(temperature=INF), ARG),
    (dict(top_k=-1), ARG), (dict(top_p=0.0), ARG), (dict(top_p=1.01), ARG), (dict(top_p=NAN), ARG),
    (dict(min_p=-0.1), ARG), (dict(min_p=1.01), ARG), (dict(min_p=NAN), ARG),
    (dict(softcap=-1.0), ARG), (dict(softcap=INF), ARG), (dict(softcap=NAN), ARG),
    (dict(temperature=Buf(10 * M), top_k=Buf(11 * M), top_p=Buf(12 * M), min_p=Buf(13 * M)), OK),
    (dict(temperature=Buf(4 * M)), ARG), (dict(top_p=Buf(10 * M + 2)), UNSUP),
]


@pytest.mark.parametrize("kw,want", SETTINGS + [
    ({}, OK), (dict(logp=None), OK), (dict(N=0, logits=None, uniforms=None, tokens=None), OK),
    (dict(dtype=torch.bfloat16), OK), (dict(N=-1), ARG), (dict(N=1 << 31), ARG), (dict(V=0), ARG),
    (dict(V=(1 << 24) + 1), ARG), (dict(logits=None), ARG), (dict(uniforms=None), ARG),
    (dict(tokens=None), ARG), (dict(ld_logits=99), ARG), (dict(tokens=Buf(M)), ARG),
    (dict(logp=Buf(4 * M)), ARG), (dict(N=1 << 22, tokens=Buf(1 << 50), logp=None, uniforms=Buf(1 << 52),
                                        workspace=Buf(1 << 54, 512)), UNSUP),
    (dict(logits=Buf(M + 2)), UNSUP), (dict(tokens=Buf(4 * M + 4)), UNSUP),
    (dict(workspace=None), WS), (dict(workspace=Buf(8 * M, 255)), WS), (dict(workspace=Buf(8 * M + 1, 512)), WS),
    (dict(V=70000, workspace=Buf(8 * M, 256)), WS), (dict(workspace=Buf(M, 512)), ARG),
])
def test_sample_logits(kw, want):
    a = dict(logits=Buf(M), uniforms=Buf(3 * M), N=3, V=100, tokens=Buf(4 * M), logp=Buf(5 * M),
             workspace=Buf(8 * M, 512))
    a.update(kw)
    assert m.flce_sample_logits_check_args(**a) == want


@pytest.mark.parametrize("kw,want", SETTINGS + [
    ({}, OK), (dict(logp=None), OK), (dict(N=0, h=None, uniforms=None, tokens=None), OK),
    (dict(dtype=torch.float32), OK), (dict(W=None), ARG), (dict(h=None), ARG), (dict(H=0), ARG),
    (dict(V=(1 << 24) + 1), ARG), (dict(N=-1), ARG), (dict(tokens=None), ARG), (dict(uniforms=None), ARG),
    (dict(tokens=Buf(2 * M)), ARG), (dict(workspace=Buf(M, 1 << 16)), ARG), (dict(h=Buf(M + 1)), UNSUP),
    (dict(workspace=None), WS), (dict(workspace=Buf(8 * M, 1000)), WS), (dict(workspace=Buf(8 * M + 4, 1 << 16)), WS),
])
def test_sample(kw, want):
    a = dict(h=Buf(M), W=Buf(2 * M), uniforms=Buf(3 * M), N=3, H=16, V=100, tokens=Buf(4 * M),
             logp=Buf(5 * M), workspace=Buf(8 * M, 1 << 16))
    a.update(kw)
    assert m.flce_sample_check_args(**a) == want


def test_workspaces():
    bf, f32 = torch.bfloat16, torch.float32
    for N, V in ((1, 100), (700, 200000), (1 << 20, 300), (5, 1 << 24), (1 << 30, 1 << 24)):
        assert 0 < m.flce_sample_workspace_size(N, 64, V, bf) <= 512 << 20
        assert 0 < m.flce_sample_logits_workspace_size(N, V, f32) <= (64 << 20) + 256
    for bad in ((-1, 8, 8), (1, 0, 8), (1, 8, 0), (1, 8, (1 << 24) + 1)):
        assert m.flce_sample_workspace_size(*bad, bf) == 0
        assert m.flce_linear_backward_workspace_size(*bad, bf) == 0
    assert m.flce_sample_logits_workspace_size(-1, 8, f32) == 0
    assert m.flce_sample_logits_workspace_size(1, 0, f32) == 0
    assert m.flce_linear_backward_workspace_size(8192, 4096, 4096, bf) >= 8192 * 4096 * 2
    assert m.flce_linear_backward_workspace_size(0, 8, 8, f32) > 0


# ---- the wrappers ----------------------------------------------------------------------------


@pytest.fixture()
def plain(monkeypatch):
    def keep(shape, seed, offset, step):
        g = torch.Generator().manual_seed(seed * 1000 + offset + (0 if step is None else int(step)))
        return (torch.rand(shape, generator=g) >= 0.5).float() * 2

    def dropout(x, residual=None, *, p, seed, offset=0, step=None, out=None):
        y = x * keep(x.shape, seed, offset, step)
        return y if residual is None else y + residual

    def norm(x, weight, residual=None, *, p, seed, offset=0, step=None, eps=1e-6, weight_offset=0.0):
        s = dropout(x, residual, p=p, seed=seed, offset=offset, step=step)
        q = torch.rsqrt((s * s).mean(1) + eps)
        return s * q[:, None] * (weight + weight_offset), s, q

    def norm_backward(dy, s, weight, rstd, ds=None, *, weight_offset=0.0, want_dresidual=True,
                      want_dweight=True, **mask):
        n, g = s * rstd[:, None], dy * (weight + weight_offset)
        d = rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
        d = d if ds is None else d + ds
        return dropout(d, **mask), d if want_dresidual else None, (dy * n).sum(0) if want_dweight else None

    def linear(x, weight, bias=None, residual=None, *, activation="none", save_slope=False):
        z = x @ weight.T + (0 if bias is None else bias)
        q = torch.sigmoid(z)
        y = z * q if activation == "silu" else z
        return (y if residual is None else y + residual,
                q * (1 + z * (1 - q)) if activation == "silu" and save_slope else None)

    def linear_backward(dy, x, weight, slope=None, *, bias=True, want_dx=True, want_dweight=True):
        dz = dy if slope is None else dy * slope
        return (dz @ weight if want_dx else None, dz.T @ x if want_dweight else None,
                dz.sum(0) if bias else None)
    monkeypatch.setattr(_dropout, "flce_dropout", dropout)
    monkeypatch.setattr(_dropout, "flce_dropout_norm", norm)
    monkeypatch.setattr(_dropout, "flce_dropout_norm_backward", norm_backward)
    monkeypatch.setattr(_linear, "flce_linear", linear)
    monkeypatch.setattr(_linear, "flce_linear_backward", linear_backward)
    return keep


@pytest.mark.parametrize("shape", [(3, 8), (2, 3, 8)])
def test_wrappers_gradients(plain, shape):
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float32).requires_grad_()  # noqa: E731
    x, res, w, b, nw = r(*shape), r(*shape), r(8, 8), r(8), r(8)
    mask = m.DropoutMask(0.5, 3, 1)

    def step():
        y, s = m.fused_dropout_norm(x, nw, mask, res)
        t = m.fused_linear(y, w, b, y, activation="silu")
        return (m.fused_dropout(t, m.DropoutMask(0.5, 4), s) ** 2).sum()

    def want():
        k = plain((x.numel() // 8, 8), 3, 1, None).reshape(shape)
        s = x * k + res
        y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6) * nw
        t = torch.nn.functional.silu(y @ w.T + b) + y
        return ((t * plain((x.numel() // 8, 8), 4, 0, None).reshape(shape) + s) ** 2).sum()
    leaves = (x, res, w, b, nw)
    got = torch.autograd.grad(step(), leaves)
    ref = torch.autograd.grad(want(), leaves)
    for a, c in zip(got, ref):
        assert torch.allclose(a, c, rtol=1e-4, atol=1e-4)


def test_wrappers_results_may_be_changed_in_place(plain):
    x = torch.randn(3, 8, requires_grad=True)
    w = torch.randn(8, 8, requires_grad=True)
    y = m.fused_linear(x, w, activation="silu")
    y *= 2
    d = m.fused_dropout(y, m.DropoutMask(0.5, 1))
    d += 1
    n, s = m.fused_dropout_norm(d, torch.ones(8), m.DropoutMask(0.5, 2))
    n *= 3
    (n.sum() + s.sum()).backward()
    assert torch.isfinite(x.grad).all() and torch.isfinite(w.grad).all()


def test_a_step_that_changed_is_refused(plain):
    x = torch.randn(3, 8, requires_grad=True)
    step = torch.zeros((), dtype=torch.int64)
    y = m.fused_dropout(x, m.DropoutMask(0.5, 1, 0, step))
    step += 1
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()


def test_second_derivatives_are_refused(plain):
    x = torch.randn(3, 8, requires_grad=True)
    w = torch.randn(8, 8, requires_grad=True)
    dx, = torch.autograd.grad(m.fused_linear(x, w, activation="silu").sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_only_on_a_gpu_and_shapes():
    x, w = torch.randn(3, 8), torch.randn(8, 8)
    for bad in (lambda: m.flce_dropout(x, p=0.5, seed=0), lambda: m.flce_linear(x, w),
                lambda: m.flce_linear_backward(x, x, w), lambda: m.flce_sample_logits(x, x[:, 0]),
                lambda: m.flce_sample(x, w, x[:, 0]), lambda: m.flce_dropout_norm(x, w[0], p=0.5, seed=0),
                lambda: m.flce_dropout_norm_backward(x, x, w[0], x[:, 0], p=0.5, seed=0),
                lambda: m.fused_linear(x, w[:, :4]), lambda: m.fused_linear(x, w, residual=x[:2]),
                lambda: m.fused_linear(x, w, activation="swish"),
                lambda: m.fused_dropout(x, m.DropoutMask(0.5, 0), x[:2]),
                lambda: m.HeadTransform(8, activation="nothing")):
        with pytest.raises(ValueError):
            bad()
