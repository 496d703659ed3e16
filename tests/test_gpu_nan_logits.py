"""Logits of NaN reach every sum of their row: a row of NaN, and a table of which some
rows are NaN, of whole tiles too."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


def make(N, V, dt):
    g = torch.Generator().manual_seed(N + V)
    W = (0.3 * torch.randn(V, 64, generator=g)).to(dt).cuda()
    h = torch.randn(N, 64, generator=g).to(dt).cuda()
    return h, W, torch.randint(0, V, (N,), generator=g).cuda()


SIZES = [(1, 700, BF), (40, 5000, BF), (140, 700, BF), (140, 40000, BF), (1100, 5000, BF),
         (3, 700, F), (70, 5000, F)]


@pytest.mark.parametrize("N,V,dt", SIZES)
@pytest.mark.parametrize("K", [0, 1, 6])
def test_a_row_of_nan(N, V, dt, K):
    import lm_head_linear_amd as m
    h, W, y = make(N, V, dt)
    clean = m.flce_logprobs(h, W, y, top_k=K)
    h[N // 2] = float("nan")
    r = m.flce_logprobs(h, W, y, top_k=K)
    keep = torch.arange(N, device="cuda") != N // 2
    assert all(bool(t[N // 2].isnan()) for t in r[:3])
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(r, clean))
    assert bool((r.top_ids[N // 2] == -1).all())


@pytest.mark.parametrize("N,V,dt", SIZES)
@pytest.mark.parametrize("rows", [(0, 1), (0, 64), (64, 128), (0, 256), (256, 512), (300, 301)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_rows_of_the_table_that_are_nan(N, V, dt, rows, cap):
    import lm_head_linear_amd as m
    h, W, y = make(N, V, dt)
    W[rows[0]:rows[1]] = float("nan")
    for K in (0, 1, 6):
        r = m.flce_logprobs(h, W, y, softcap=cap, top_k=K)
        assert all(bool(t.isnan().all()) for t in r[:3]), K
        z = h.float() @ W.float().t()
        z[:, rows[0]:rows[1]] = -torch.inf
        if K:
            assert not bool(((r.top_ids >= rows[0]) & (r.top_ids < rows[1])).any())
            best = z.gather(1, r.top_ids[:, :1])[:, 0]
            assert bool((best >= z.max(1).values - 1e-3).all())
