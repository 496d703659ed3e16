"""TiedLMHead.sample with tensors of the caller for its results: they get them, or the call
is refused (no GPU: plain torch in the library call's place)."""
import pytest
import torch

import lm_head_linear_amd as m


@pytest.fixture()
def head(monkeypatch):
    """A head whose rows are x itself and whose tokens are the rows' largest logits."""
    def sample(h, W, uniforms, *, tokens=None, logp=None, workspace=None, temperature=1.0, softcap=0.0):
        for name, t, dt in (("uniforms", uniforms, torch.float32), ("tokens", tokens, torch.int64),
                            ("logp", logp, torch.float32), ("temperature", temperature, torch.float32)):
            if isinstance(t, torch.Tensor) and (t.shape != h.shape[:1] or t.dtype != dt or not t.is_contiguous()):
                raise ValueError(f"{name} must be {h.shape[0]} contiguous {dt}")
        assert workspace is None or workspace.dtype == torch.uint8
        tokens = torch.empty(h.shape[0], dtype=torch.int64) if tokens is None else tokens
        logp = torch.empty(h.shape[0]) if logp is None else logp
        z = h @ W.T
        tokens.copy_(z.argmax(1))
        logp.copy_(torch.log_softmax(z, 1).amax(1))
        return m.Sampled(tokens, logp)
    monkeypatch.setattr(m, "flce_sample", sample)
    t = m.TiedLMHead(11, 8)
    monkeypatch.setattr(t, "rows", lambda x, residual=None: x)
    return t


@pytest.mark.parametrize("shape", [(4,), (4, 1), (2, 3)])
def test_results_reach_the_callers_tensors(head, shape):
    x, u = torch.randn(*shape, 8), torch.rand(shape)
    want = head.sample(x, u)
    tokens, logp = torch.full(shape, -7), torch.full(shape, -7.0)
    r = head.sample(x, u, tokens=tokens, logp=logp, workspace=torch.empty(256, dtype=torch.uint8),
                    temperature=torch.ones(shape).expand(*shape))
    assert r.tokens.data_ptr() == tokens.data_ptr() and r.logp.data_ptr() == logp.data_ptr()
    for a, b, c in zip(r, want, (tokens, logp)):
        assert a.shape == shape and torch.equal(a, b) and torch.equal(c, b)


@pytest.mark.parametrize("name,dt", [("tokens", torch.int64), ("logp", torch.float32)])
def test_a_column_of_a_table_is_refused(head, name, dt):
    """A column's elements lie apart: the results went to a copy of it, unseen."""
    x, u = torch.randn(4, 8), torch.rand(4)
    table = torch.full((4, 10), -7, dtype=dt)
    with pytest.raises(ValueError, match=f"{name} must be contiguous"):
        head.sample(x, u, **{name: table[:, 3]})
    with pytest.raises(ValueError):
        head.sample(x, u, **{name: torch.full((5,), -7, dtype=dt)})
    assert bool((table == -7).all())


def test_settings_may_have_any_strides(head):
    x, u = torch.randn(2, 3, 8), torch.rand(3, 2).T
    r = head.sample(x, u, temperature=torch.ones(()).expand(2, 3))
    assert r.tokens.shape == (2, 3)
