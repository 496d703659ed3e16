"""Sampling from a head of few ids with more rows than one grid takes: each row is what it
is alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,dt", [(7, torch.bfloat16), (1, torch.float32)])
def test_more_rows_than_a_grid_takes(V, dt):
    import lm_head_linear_amd as m
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    most = (2 ** 32 - 1) // 1024
    N, H = most + 77, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    # whole numbers: the logits are exact, whichever kernel forms them
    h = torch.randint(-3, 4, (N, H), generator=g, device="cuda").to(dt)
    W = torch.randint(-2, 3, (V, H), generator=g, device="cuda").to(dt)
    u = torch.rand(N, generator=g, device="cuda")
    T = 0.5 + torch.rand(N, generator=g, device="cuda")
    r = m.flce_sample(h, W, u, temperature=T, top_k=5)
    assert bool(((r.tokens >= 0) & (r.tokens < V)).all())
    for part in (slice(0, 50), slice(most - 40, most + 40), slice(N - 20, N)):
        p = m.flce_sample(h[part].contiguous(), W, u[part].contiguous(),
                          temperature=T[part].contiguous(), top_k=5)
        assert torch.equal(p.tokens, r.tokens[part]) and torch.equal(p.logp, r.logp[part])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [49151, 49152, 49153])
def test_either_side_of_the_maxima(V, dt):
    """Up to 64 rows from 49152 logits on have the maxima of their parts formed first: the
    same rows among more than 64 have not."""
    import lm_head_linear_amd as m
    from tests.test_gpu_sample import compare, make, run
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert (m.flce_sample_logits_workspace_size(64, V, dt) > 256) == (V >= 49152)
    assert m.flce_sample_logits_workspace_size(65, V, dt) == 256
    z, u = make(65, V, dt, V, masked=0.2)
    for kw in (dict(T=0.7, k=50, p=0.9), dict(T=0.0), dict(k=3, cap=20.0), dict(T=1.2, k=900)):
        some, all_ = run(z[:64], u[:64], **kw), run(z, u, **kw)
        assert torch.equal(some.tokens, all_.tokens[:64]) and torch.equal(some.logp, all_.logp[:64])
        compare(run(z[:2], u[:2], **kw), z[:2], u[:2], **kw)
