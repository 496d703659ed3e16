"""What the autograd forms return may be changed in place, as the results of torch's own
operations may: the wrappers around the GPU calls, run on the CPU with plain torch in
the calls' place."""
import pytest
import torch

import lm_head_linear_amd as m
from lm_head_linear_amd import _ops


@pytest.fixture(autouse=True)
def plain_calls(monkeypatch):
    def embedding(tokens, W, *, scale=1.0, padding_index=-100):
        return scale * W[tokens.clamp_min(0)] * (tokens != padding_index)[:, None]

    def embedding_backward(tokens, dout, V, *, scale=1.0, padding_index=-100, **kw):
        live = tokens != padding_index
        return torch.zeros(V, dout.shape[1]).index_add(0, tokens[live], scale * dout[live])

    def norm(x, weight, residual=None, *, eps=1e-6, weight_offset=0.0):
        s = x if residual is None else x + residual
        q = torch.rsqrt((s * s).mean(1) + eps)
        return s * q[:, None] * (weight + weight_offset), s, q

    def norm_backward(dy, s, weight, rstd, ds=None, *, weight_offset=0.0, want_dweight=True):
        n, g = s * rstd[:, None], dy * (weight + weight_offset)
        dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
        return dx if ds is None else dx + ds, (dy * n).sum(0)
    monkeypatch.setattr(_ops, "flce_embedding", embedding)
    monkeypatch.setattr(_ops, "flce_embedding_backward", embedding_backward)
    monkeypatch.setattr(_ops, "flce_rms_norm", norm)
    monkeypatch.setattr(_ops, "flce_rms_norm_backward", norm_backward)


def grads(f, *leaves):
    for t in leaves:
        t.grad = None
    f().backward()
    return [t.grad.clone() for t in leaves]


@pytest.mark.parametrize("shape", [(7,), (2, 3), (2, 3, 4), ()])
def test_a_lookup_changed_in_place(shape):
    torch.manual_seed(0)
    W = torch.randn(9, 5, requires_grad=True)
    t = torch.randint(0, 9, shape)
    pos, c = torch.randn(*shape, 5), torch.randn(*shape, 5)

    def there():
        e = m.fused_embedding(t, W, scale=1.5)
        assert e.shape == (*shape, 5)
        e += pos
        e.mul_(2)
        return (torch.tanh(e) * c).sum()

    def beside():
        return (torch.tanh(2 * (1.5 * W[t] + pos)) * c).sum()
    (a,), (b,) = grads(there, W), grads(beside, W)
    assert torch.allclose(a, b, atol=1e-5)


@pytest.mark.parametrize("shape", [(5,), (6, 5), (2, 3, 5)])
@pytest.mark.parametrize("residual", [False, True])
def test_a_norm_changed_in_place(shape, residual):
    torch.manual_seed(1)
    x = torch.randn(*shape, requires_grad=True)
    r = torch.randn(*shape, requires_grad=True)
    w = torch.randn(5, requires_grad=True)
    c, d = torch.randn(*shape), torch.randn(*shape)

    def there():
        if not residual:
            y = m.fused_rms_norm(x, w)
            y *= 3
            return (y * c).sum()
        y, s = m.fused_rms_norm(x, w, r)
        assert y.shape == s.shape == shape
        y += 1
        y *= 3
        return (y * c).sum() + (torch.sin(s) * d).sum()

    def beside():
        s = x + r if residual else x
        y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6) * w
        if not residual:
            return (3 * y * c).sum()
        return (3 * (y + 1) * c).sum() + (torch.sin(s) * d).sum()
    leaves = (x, r, w) if residual else (x, w)
    for a, b in zip(grads(there, *leaves), grads(beside, *leaves)):
        assert torch.allclose(a, b, atol=1e-5)


def test_the_residual_stream_changed_in_place():
    """The norm's backward reads s: changed before it, autograd says so; where only the
    sum is used, it may be changed."""
    x = torch.randn(3, 5, requires_grad=True)
    r = torch.randn(3, 5, requires_grad=True)
    w = torch.randn(5, requires_grad=True)
    y, s = m.fused_rms_norm(x, w, r)
    s += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (y.sum() + s.sum()).backward()
    y, s = m.fused_rms_norm(x, w, r)
    with torch.no_grad():
        t = s.detach().clone()
    s = s.clone()
    s += y
    s.sum().backward()
    assert x.grad is not None and torch.equal(x.grad, r.grad) and t.shape == s.shape


def test_gradients_of_the_two_inputs_are_tensors_of_their_own():
    """x and the residual get the same values: leaves that both keep them do not share
    their memory, whether the norm, the sum or both were used."""
    for use in ("y", "s", "both"):
        x = torch.randn(2, 3, 5, requires_grad=True)
        r = torch.randn(2, 3, 5, requires_grad=True)
        y, s = m.fused_rms_norm(x, torch.ones(5), r)
        sum({"y": [y.sin().sum()], "s": [s.cos().sum()], "both": [y.sum(), s.sum()]}[use]).backward()
        assert torch.equal(x.grad, r.grad)
        x.grad += 1
        assert not torch.equal(x.grad, r.grad)
