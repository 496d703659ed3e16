"""Tables and rows without elements are the library's argument error, not an error of the
binding, which has no workspace to pass for them."""
import pytest
import torch

import lm_head_linear_amd as m
from lm_head_linear_amd import _lib, _ops


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    """The checks come before any GPU work: they run on tensors of the CPU."""
    monkeypatch.setattr(_ops, "_on_gpu", lambda where, dev: None)
    monkeypatch.setattr(_ops, "_stream", lambda dev: None)

    def run(where, dev, fn, *args):
        rc = fn(*args)
        assert rc != _lib.OK, "nothing may be launched here"
        raise m.FlceError(rc, where)
    monkeypatch.setattr(_ops, "_run", run)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,V", [(8, 0), (0, 5), (0, 0)])
@pytest.mark.parametrize("N", [0, 4])
def test_empty_tables(dt, H, V, N):
    h, W, y = torch.zeros(N, H, dtype=dt), torch.zeros(V, H, dtype=dt), torch.zeros(N).long()
    lse = torch.zeros(N)
    calls = [lambda: m.flce_logprobs(h, W, y, top_k=2), lambda: m.flce_logprobs(h, W),
             lambda: m.flce_logprobs_backward(h, W, y, lse, lse, lse, lse),
             lambda: m.flce_embedding(y, W), lambda: m.flce_embedding_backward(y, h, V)]
    if H == 0:
        w = torch.zeros(0, dtype=dt)
        calls += [lambda: m.flce_rms_norm(h, w), lambda: m.flce_rms_norm_backward(h, h, w, lse)]
    for call in calls:
        with pytest.raises(m.FlceError) as e:
            call()
        assert e.value.code == _lib.ERR_ARG


def test_bf16_gradients_of_float32_rows_are_unsupported():
    h, W, y, lse = torch.zeros(4, 8), torch.zeros(5, 8), torch.zeros(4).long(), torch.zeros(4)
    with pytest.raises(m.FlceError) as e:
        m.flce_logprobs_backward(h, W, y, lse, None, lse, grad_dtype=torch.bfloat16)
    assert e.value.code == _lib.ERR_UNSUPPORTED
