"""A row's values do not depend on the rows beside it: within each of the kernels (bf16
with up to 128 rows, bf16 tiles, float32) the same row gives the same bits in calls of
any count of rows, over vocabularies of a few tiles and of hundreds."""
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


CASES = [(70000, BF, 128, (1, 5, 16, 17, 33, 49, 65)),
         (999, BF, 128, (1, 17, 33, 49, 65)),
         (70000, BF, 4200, (129, 700, 1025, 4097)),
         (20000, BF, 4200, (129, 300, 1025, 4097)),
         (2001, BF, 4200, (129, 300, 1025, 4097)),
         (5003, F, 300, (1, 20, 33, 64, 257)),
         (33001, F, 129, (1, 64, 128))]


@pytest.mark.parametrize("V,dt,most,counts", CASES)
@pytest.mark.parametrize("K", [0, 1, 5, 17])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_the_same_bits_for_any_count_of_rows(V, dt, most, counts, K, cap):
    import lm_head_linear_amd as m
    g = torch.Generator().manual_seed(V)
    W = (0.2 * torch.randn(V, 64, generator=g)).to(dt).cuda()
    h = torch.randn(most, 64, generator=g).to(dt).cuda()
    y = torch.randint(0, V, (most,), generator=g).cuda()
    kw = dict(softcap=cap, temperature=0.9, top_k=K)
    whole = m.flce_logprobs(h, W, y, **kw)
    assert bool((whole.logp < 0).all()) and bool((whole.entropy > 0).all())
    for n in counts:
        part = m.flce_logprobs(h[:n], W, y[:n], **kw)
        for name, a, b in zip(whole._fields, whole, part):
            assert torch.equal(a[:n], b), (n, name, int((a[:n] != b).sum()))


def test_the_last_rows_of_a_long_call():
    """More rows than one chunk holds, over hundreds of tiles: those of the short last
    chunk have the bits of a call of their own."""
    import lm_head_linear_amd as m
    g = torch.Generator().manual_seed(2)
    N, V = 8192 + 200, 70000
    W = (0.2 * torch.randn(V, 64, generator=g)).bfloat16().cuda()
    h = torch.randn(N, 64, generator=g).bfloat16().cuda()
    y = torch.randint(0, V, (N,), generator=g).cuda()
    whole = m.flce_logprobs(h, W, y, top_k=5)
    last = m.flce_logprobs(h[8192:], W, y[8192:], top_k=5)
    first = m.flce_logprobs(h[:300], W, y[:300], top_k=5)
    assert all(torch.equal(a[8192:], b) for a, b in zip(whole, last))
    assert all(torch.equal(a[:300], b) for a, b in zip(whole, first))


def test_many_rows_over_millions_of_ids():
    """The logits of 100 rows over a vocabulary of more than 2^21 ids (844 MB) and of 128
    over 2^22 (2 GiB) with alternatives, next to the first rows alone."""
    import lm_head_linear_amd as m
    g = torch.Generator().manual_seed(1)
    for N, V in ((100, 2200001), (128, 4194304)):
        W = torch.randn(V, 8, generator=g).bfloat16().cuda()
        h = torch.randn(N, 8, generator=g).bfloat16().cuda()
        y = torch.randint(0, V, (N,), generator=g).cuda()
        whole = m.flce_logprobs(h, W, y, top_k=3)
        for n in (1, 40):
            part = m.flce_logprobs(h[N - n:], W, y[N - n:], top_k=3)
            assert all(torch.equal(a[N - n:], b) for a, b in zip(whole, part))
        x = h[-1].double() @ W.double().t()
        assert abs(float(whole.lse[-1]) - float(torch.logsumexp(x, 0))) < 1e-4
        assert bool((x[whole.top_ids[-1]] >= x.topk(3).values.min() - 1e-4).all())
