"""Log probabilities of tokens that hold nearly all of the probability, at logits far
from zero.

The logits are single bf16 values (one column of h is 1, the rest 0), so z is exact. The
largest term of the sum is exactly 1, so S >= 1 and no log probability is above zero, and
a small one is off by
 - 2^-24 for each of at most 40 additions whose sum is in [1, 2): 40 u;
 - of itself, the errors of the small terms: their x are rounded (u |x| each, two of
   them, twice that with the rounded 1 / T), x - M and its product with log2 e (2 u |x - M|
   with |x - M| <= 40), the hardware exp2 (2^-22) and at most 100 additions: 4 u |x| + 2e-5."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


def peaked(N, V, top, dt, seed=0):
    """One logit at `top`, the others 12 to 22 below it, on steps that bf16 holds."""
    g = torch.Generator().manual_seed(seed)
    z = top - 12 - 2 * torch.randint(0, 6, (V,), generator=g).float()
    at = int(torch.randint(0, V, (1,), generator=g))
    z[at] = top
    assert torch.equal(z.to(BF).float(), z)
    h, W = torch.zeros(N, 64), torch.zeros(V, 64)
    h[:, 5], W[:, 5] = 1, z
    return h.to(dt).cuda(), W.to(dt).cuda(), torch.full((N,), at, device="cuda"), z.double().cuda()


@pytest.mark.parametrize("N,dt", [(1, BF), (3, BF), (40, BF), (130, BF), (2, F), (70, F)])
@pytest.mark.parametrize("V", [700, 9000])
@pytest.mark.parametrize("T", [1.0, 0.7])
@pytest.mark.parametrize("top", [-22.0, 40.0, 296.0])
def test_a_small_log_probability_is_kept(N, dt, V, T, top):
    import lm_head_linear_amd as m
    h, W, y, z = peaked(N, V, top, dt, seed=V)
    r = m.flce_logprobs(h, W, y, temperature=T, top_k=3)
    x = z / T
    want = float(x.max() - torch.logsumexp(x, 0))
    assert -0.1 < want < 0
    bound = 40 * U + abs(want) * (4 * U * float(x.abs().max()) + 2e-5)
    err = (r.logp.double() - want).abs().max()
    assert float(err) <= bound, (float(err), bound, want)
    assert bool((r.logp <= 0).all())
    assert torch.equal(r.top_logp[:, 0], r.logp) and bool((r.top_ids[:, 0] == y).all())


@pytest.mark.parametrize("N,dt", [(100, BF), (600, BF), (200, F)])
@pytest.mark.parametrize("cap,T", [(0.0, 1.0), (0.0, 0.3), (50.0, 0.25), (30.0, 1.3)])
def test_no_log_probability_is_above_zero(N, dt, cap, T):
    """Rows whose best token holds from little to all of the probability."""
    import lm_head_linear_amd as m
    g = torch.Generator().manual_seed(N)
    W = torch.randn(3000, 96, generator=g).to(dt).cuda()
    y = torch.randint(0, 3000, (N,), generator=g).cuda()
    h = W[y] * (2 * torch.rand(N, 1, generator=g)).to(dt).cuda()
    r = m.flce_logprobs(h, W, y, softcap=cap, temperature=T, top_k=4)
    assert bool((r.logp <= 0).all()) and bool((r.top_logp <= 0).all())
    best = r.top_ids[:, 0] == y
    assert int(best.sum()) > N // 4
    assert torch.equal(r.top_logp[best, 0], r.logp[best])
