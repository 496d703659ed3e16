"""What the bf16 gradients of log probabilities lose to rounding: the stored gradients, to
half a step once, and G of the ids that are not given, to half a step of each. The given
tokens' G, the largest of their rows, loses nothing, neither in dH nor in dW.

Both losses are formed here in float64 from the definition: r by rounding the exact
gradients, g by rounding the other ids' G before the products. They are independent, so the
norm of the error is that of (r, g) to within a few percent at the 2000 elements and more
here; the float32 logits (2^-20 of them), exponents and sums add 2^-13 of G at most to
single elements and a hundredth of that to a norm of such many: 2^-14."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


def loss(x, exact):
    return float((x - exact).norm() / exact.norm())


CASES = [(40, 64, 300), (128, 133, 700), (300, 72, 1001), (600, 256, 300), (1000, 512, 2000),
         (3000, 128, 9000), (700, 64, 70000), (2500, 1024, 1500), (40000, 16, 300), (70000, 8, 200)]


@pytest.mark.parametrize("N,H,V", CASES)
@pytest.mark.parametrize("common", [0.0, 4.0])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("chunk", ["0", "512"])
def test_only_the_other_ids_and_the_stores_are_rounded(N, H, V, common, accumulate, chunk,
                                                       monkeypatch):
    """Also with a component that all rows of W share, which G's sum of 0 takes out of dH."""
    import lm_head_linear_amd as m
    monkeypatch.setenv("FLCE_VCHUNK", chunk)
    g = torch.Generator().manual_seed(N + V)
    std = 1.3 / math.sqrt(H)
    W = std * torch.randn(V, H, generator=g) + common * std * torch.randn(1, H, generator=g)
    W = W.bfloat16().cuda()
    y = torch.randint(0, V, (N,), generator=g).cuda()
    y[::9] = IGN
    h = torch.randn(N, H, generator=g).bfloat16().cuda()
    a = torch.randn(N, generator=g).cuda()
    r = m.flce_logprobs(h, W, y)
    base = (0.3 * torch.randn(V, H, generator=g)).bfloat16().cuda() if accumulate else None
    dH, dW = m.flce_logprobs_backward(h, W, y, r.lse, None, a,
                                      dW=None if base is None else base.clone(),
                                      accumulate_dW=accumulate)
    x = h.double() @ W.double().t()
    live, at = y != IGN, y.clamp_min(0)[:, None]
    hot = torch.zeros_like(x).scatter_(1, at, 1.0)
    G = a.double()[:, None] * (hot - torch.softmax(x, 1)) * live[:, None]
    rounded = torch.where(hot > 0, G, G.float().bfloat16().double())
    for name, got, exact, less in (
            ("dH", dH, G @ W.double(), rounded @ W.double()),
            ("dW", dW, G.t() @ h.double() + (0 if base is None else base.double()),
             rounded.t() @ h.double() + (0 if base is None else base.double()))):
        bound = 1.05 * math.hypot(loss(exact.bfloat16().double(), exact), loss(less, exact)) + 2.0 ** -14
        assert loss(got.double(), exact) <= bound, (name, loss(got.double(), exact), bound)
