"""What the autograd forms return may be changed in place: a lookup, a norm and log
probabilities so changed give the bits of the same step out of place."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(30,), (2, 70)])
def test_a_step_in_place(dt, shape):
    import lm_head_linear_amd as m
    torch.manual_seed(3)
    t = m.TiedLMHead(300, 48, embed_scale=2.0, device="cuda", dtype=dt)
    x, y = torch.randint(0, 300, shape, device="cuda"), torch.randint(0, 300, shape, device="cuda")
    pos = torch.randn(*shape, 48, device="cuda").to(dt)
    c = torch.randn(shape, device="cuda")

    def step(inplace):
        t.zero_grad(set_to_none=True)
        e = t.embed(x)
        if inplace:
            e += pos
        else:
            e = e + pos
        n = t.norm(torch.tanh(e), residual=e)
        if inplace:
            n *= 2
        else:
            n = n * 2
        r = m.token_logprobs(n, y, t.weight, top_k=2)
        logp = r.logp
        if inplace:
            logp *= c
            logp += 1
        else:
            logp = logp * c + 1
        (logp.sum() + 0.1 * r.entropy.sum()).backward()
        return [logp.detach().clone(), t.weight.grad.clone(), t.norm_weight.grad.clone()]
    assert all(torch.equal(a, b) for a, b in zip(step(True), step(False)))
