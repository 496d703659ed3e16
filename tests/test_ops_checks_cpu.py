"""The refusals of the operators around the head (no GPU): every rule of their
check_args entries, which run the checks of the calls themselves."""
import os

import pytest
import torch

import lm_head_linear_amd as m
from lm_head_linear_amd import _lib

OK, ARG, UNSUP, WS = _lib.OK, _lib.ERR_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_WORKSPACE


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


M = 1 << 20


def norm(**kw):
    a = dict(x=Buf(M), weight=Buf(2 * M), residual=Buf(3 * M), N=4, H=24, y=Buf(4 * M),
             s=Buf(5 * M), rstd=Buf(6 * M))
    a.update(kw)
    return m.flce_rms_norm_check_args(**a)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(N=0, x=None, y=None, residual=None, s=None, rstd=None), OK),
    (dict(rstd=None), OK), (dict(residual=None, s=None), OK),
    (dict(y=Buf(M)), OK), (dict(s=Buf(3 * M)), OK), (dict(s=Buf(M)), OK),
    (dict(weight_dtype=torch.float32), OK), (dict(dtype=torch.float32), OK),
    (dict(x=Buf(M + 2)), OK), (dict(eps=0.0), OK),
    (dict(N=-1), ARG), (dict(N=1 << 31), ARG), (dict(H=0), ARG), (dict(H=(1 << 24) + 1), ARG),
    (dict(x=None), ARG), (dict(y=None), ARG), (dict(weight=None), ARG),
    (dict(residual=None), ARG), (dict(s=None), ARG),
    (dict(eps=-1e-6), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(weight_offset=float("nan")), ARG),
    (dict(ld_x=23), ARG), (dict(ld_y=23), ARG), (dict(ld_s=0), ARG), (dict(ld_res=(1 << 31) + 1), ARG),
    (dict(y=Buf(M), s=Buf(M)), ARG), (dict(y=Buf(M + 48)), ARG), (dict(y=Buf(M), ld_y=25), ARG),
    (dict(s=Buf(3 * M + 2)), ARG), (dict(y=Buf(3 * M)), ARG), (dict(y=Buf(5 * M)), ARG),
    (dict(y=Buf(2 * M)), ARG), (dict(rstd=Buf(M)), ARG), (dict(rstd=Buf(4 * M + 4)), ARG),
    (dict(dtype=torch.float32, weight_dtype=torch.bfloat16), UNSUP),
    (dict(x=Buf(M + 1)), UNSUP), (dict(rstd=Buf(6 * M + 2)), UNSUP),
])
def test_rms_norm(kw, want):
    assert norm(**kw) == want


def norm_bwd(**kw):
    a = dict(dy=Buf(M), s=Buf(2 * M), weight=Buf(3 * M), rstd=Buf(4 * M), ds=Buf(5 * M), N=4, H=24,
             dx=Buf(6 * M), dweight=Buf(7 * M), workspace=Buf(8 * M, 512))
    a.update(kw)
    return m.flce_rms_norm_backward_check_args(**a)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(ds=None), OK), (dict(dweight=None, workspace=None), OK),
    (dict(dx=Buf(M)), OK), (dict(dx=Buf(5 * M)), OK),
    (dict(dy=None), ARG), (dict(s=None), ARG), (dict(rstd=None), ARG), (dict(dx=None), ARG),
    (dict(dx=Buf(2 * M)), ARG), (dict(dx=Buf(M + 2)), ARG), (dict(dx=Buf(7 * M)), ARG),
    (dict(dweight=Buf(3 * M)), ARG), (dict(dweight=Buf(8 * M + 4)), ARG),
    (dict(workspace=Buf(M, 512)), ARG), (dict(ld_dx=3), ARG), (dict(H=-1), ARG),
    (dict(workspace=None), WS), (dict(workspace=Buf(8 * M, 383)), WS),
    (dict(workspace=Buf(8 * M + 16, 512)), WS), (dict(dweight=Buf(7 * M + 1)), UNSUP),
])
def test_rms_norm_backward(kw, want):
    assert norm_bwd(**kw) == want


def test_rms_norm_workspace():
    assert m.flce_rms_norm_backward_workspace_size(4, 24) == 512
    assert m.flce_rms_norm_backward_workspace_size(1 << 20, 4096) == 1024 * 4096 * 4
    assert m.flce_rms_norm_backward_workspace_size(0, 24) == 256
    assert m.flce_rms_norm_backward_workspace_size(-1, 24) == 0


def embed(**kw):
    a = dict(tokens=Buf(M), W=Buf(2 * M), N=4, H=24, V=10, out=Buf(3 * M), status=Buf(4 * M))
    a.update(kw)
    return m.flce_embedding_check_args(**a)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(status=None), OK), (dict(N=0, tokens=None, out=None), OK), (dict(ld_out=30), OK),
    (dict(N=-1), ARG), (dict(V=0), ARG), (dict(H=0), ARG), (dict(V=(1 << 31) + 1), ARG),
    (dict(scale=float("inf")), ARG), (dict(W=None), ARG), (dict(tokens=None), ARG),
    (dict(out=None), ARG), (dict(ld_out=23), ARG), (dict(out=Buf(2 * M)), ARG),
    (dict(out=Buf(M + 8)), ARG), (dict(status=Buf(3 * M)), ARG),
    (dict(tokens=Buf(M + 4)), UNSUP), (dict(out=Buf(3 * M + 1)), UNSUP),
])
def test_embedding(kw, want):
    assert embed(**kw) == want


def embed_bwd(**kw):
    n = m.flce_embedding_backward_workspace_size(100, 24, 10)
    a = dict(tokens=Buf(M), dout=Buf(2 * M), N=100, H=24, V=10, dW=Buf(3 * M), status=Buf(4 * M),
             workspace=Buf(5 * M, n))
    a.update(kw)
    return m.flce_embedding_backward_check_args(**a)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(grad_dtype=torch.float32), OK), (dict(accumulate_dW=True), OK),
    (dict(dW=None), ARG), (dict(dout=None), ARG), (dict(dW=Buf(2 * M)), ARG),
    (dict(workspace=Buf(3 * M, 1 << 16)), ARG), (dict(status=Buf(3 * M)), ARG),
    (dict(dtype=torch.float32, grad_dtype=torch.bfloat16), UNSUP),
    (dict(workspace=None), WS), (dict(workspace=Buf(5 * M, 1023)), WS),
    (dict(workspace=Buf(5 * M + 128, 1 << 16)), WS),
])
def test_embedding_backward(kw, want):
    assert embed_bwd(**kw) == want


def test_embedding_workspace():
    size = m.flce_embedding_backward_workspace_size
    assert size(0, 8, 8) == 256 and size(1, 8, 0) == 0
    # keys and positions, twice beyond one chunk of 1024; two partial rows for each 256
    # tokens, or 64 up to 8192
    assert size(1024, 64, 100) == 2 * 1024 * 4 + 2 * 16 * 64 * 4
    assert size(16384, 4096, 131072) == 4 * 16384 * 4 + 2 * 64 * 4096 * 4
    # 256 digit counts a block beyond what is merged at once
    assert size(1 << 15, 64, 100) == 4 * (1 << 15) * 4 + 2 * 128 * 64 * 4
    assert size(1 << 16, 64, 100) == 4 * (1 << 16) * 4 + 256 * 8 * 4 + 2 * 256 * 64 * 4


def lp(**kw):
    a = dict(h=Buf(M), W=Buf(2 * M), tokens=Buf(3 * M), N=4, H=24, V=100, top_k=3,
             logp=Buf(4 * M), entropy=Buf(5 * M), lse=Buf(6 * M), top_logp=Buf(7 * M),
             top_ids=Buf(8 * M), status=Buf(9 * M))
    a.update(kw)
    if "workspace" not in a:
        a["workspace"] = Buf(64 * M, max(1, m.flce_logprobs_workspace_size(
            a["N"], a["H"], a["V"], a.get("dtype", torch.bfloat16), a["top_k"])))
    return m.flce_logprobs_check_args(**a)


NOTOP = dict(top_k=0, top_logp=None, top_ids=None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (NOTOP, OK), (dict(entropy=None, lse=None, status=None), OK),
    (dict(tokens=None, logp=None), OK), (dict(N=1000), OK), (dict(dtype=torch.float32), OK),
    (dict(N=0, h=None, tokens=None, logp=None), OK), (dict(H=7), OK), (dict(V=1), OK),
    (dict(top_k=32), OK), (dict(temperature=0.01, softcap=30.0), OK),
    (dict(N=-1), ARG), (dict(H=0), ARG), (dict(V=0), ARG), (dict(top_k=-1), ARG),
    (dict(top_k=33), ARG), (dict(softcap=-1.0), ARG), (dict(softcap=float("inf")), ARG),
    (dict(temperature=0.0), ARG), (dict(temperature=-1.0), ARG),
    (dict(temperature=float("nan")), ARG), (dict(temperature=1e-39), ARG),
    (dict(h=None), ARG), (dict(W=None), ARG), (dict(tokens=None), ARG), (dict(logp=None), ARG),
    (dict(top_ids=None), ARG), (dict(top_logp=None), ARG), (dict(top_k=0), ARG),
    (dict(logp=Buf(5 * M)), ARG), (dict(lse=Buf(M)), ARG), (dict(top_ids=Buf(2 * M + 16)), ARG),
    (dict(status=Buf(3 * M + 4)), ARG), (dict(workspace=Buf(M, 1 << 20)), ARG),
    (dict(h=Buf(M + 8)), UNSUP), (dict(W=Buf(2 * M + 2)), UNSUP), (dict(logp=Buf(4 * M + 2)), UNSUP),
    (dict(dtype=torch.float32, h=Buf(M + 8)), OK), (dict(top_ids=Buf(8 * M + 4)), UNSUP),
    (dict(workspace=None), WS), (dict(workspace=Buf(64 * M, 1024)), WS),
    (dict(workspace=Buf(64 * M + 64, 1 << 24)), WS),
])
def test_logprobs(kw, want):
    assert lp(**kw) == want


def lp_bwd(**kw):
    a = dict(h=Buf(M), W=Buf(2 * M), tokens=Buf(3 * M), lse=Buf(4 * M), entropy=Buf(5 * M),
             grad_logp=Buf(6 * M), grad_entropy=Buf(7 * M), N=4, H=24, V=100, dH=Buf(8 * M),
             dW=Buf(9 * M), status=Buf(10 * M))
    a.update(kw)
    if "workspace" not in a:
        a["workspace"] = Buf(64 * M, max(1, m.flce_logprobs_backward_workspace_size(
            a["N"], a["H"], a["V"], a.get("dtype", torch.bfloat16), a.get("grad_dtype"))))
    return m.flce_logprobs_backward_check_args(**a)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(grad_logp=None), OK), (dict(grad_entropy=None, entropy=None), OK),
    (dict(grad_dtype=torch.float32), OK), (dict(dtype=torch.float32), OK), (dict(H=13), OK),
    (dict(N=0, h=None, dH=None, tokens=None, lse=None, entropy=None, grad_logp=None,
          grad_entropy=None), OK),
    (dict(grad_logp=None, grad_entropy=None), ARG), (dict(entropy=None), ARG),
    (dict(lse=None), ARG), (dict(tokens=None), ARG), (dict(dH=None), ARG), (dict(dW=None), ARG),
    (dict(dW=Buf(2 * M)), ARG), (dict(dH=Buf(9 * M)), ARG), (dict(dW=Buf(6 * M)), ARG),
    (dict(dH=Buf(4 * M)), ARG), (dict(workspace=Buf(9 * M, 1 << 24)), ARG),
    (dict(temperature=0.0), ARG), (dict(softcap=float("nan")), ARG), (dict(N=-2), ARG),
    (dict(dH=Buf(8 * M + 8)), UNSUP), (dict(grad_logp=Buf(6 * M + 1)), UNSUP),
    (dict(workspace=None), WS), (dict(workspace=Buf(64 * M, 4096)), WS),
])
def test_logprobs_backward(kw, want):
    assert lp_bwd(**kw) == want


def test_float32_inputs_take_no_bf16_gradients():
    assert lp_bwd(dtype=torch.float32, grad_dtype=torch.bfloat16,
                  workspace=Buf(64 * M, 1 << 24)) == UNSUP


def test_logprobs_workspace():
    size = m.flce_logprobs_workspace_size
    bf = torch.bfloat16
    assert size(4, 8, 8, bf, 33) == 0 and size(4, 0, 8, bf, 0) == 0 and size(0, 8, 8, bf, 4) == 512
    # one token: four partials for each 64 vocabulary rows, and its logits
    assert size(1, 4096, 131072, bf, 8) < 2048 * 16 + 131072 * 4 + 4096
    assert size(1, 4096, 131072, bf, 0) < 2048 * 12 + 4096
    # the candidates of a chunk of tokens stay below 1 GiB, whatever N is
    a, b = size(1 << 17, 64, 256000, bf, 32), size(1 << 18, 64, 256000, bf, 32)
    assert b - a < (1 << 17) * (64 * 2 + 32) and a < (1 << 30) + (1 << 17) * 256 + (1 << 25)


def test_sizes_beyond_one_grid():
    """A grid holds less than 2^32 threads, and 65535 workgroups along its second axis."""
    at = lambda i: Buf(i << 58)  # noqa: E731
    big = dict(tokens=at(1), W=at(2), out=at(3), status=None, H=2048)
    assert embed(**big, N=(1 << 24), V=100) == OK        # two 2 KiB pieces a row
    assert embed(**big, N=(1 << 25) + 8, V=100) == UNSUP
    back = dict(tokens=at(1), dout=at(2), dW=at(3), status=None, N=100, H=4096,
                workspace=Buf(8 << 58, 1 << 30))
    assert embed_bwd(**back, V=1 << 24) == OK            # 128 GiB of dW
    assert embed_bwd(**back, V=1 << 25) == UNSUP
    few = dict(h=at(1), W=at(2), tokens=at(3), logp=at(4), entropy=None, lse=None, status=None,
               N=1, H=8, dtype=torch.float32, **NOTOP)
    ws = lambda **k: Buf(5 << 58, m.flce_logprobs_workspace_size(  # noqa: E731
        1, 8, k["V"], torch.float32, 0))
    assert lp(**few, V=1 << 29, workspace=ws(V=1 << 29)) == OK
    assert lp(**few, V=1 << 30, workspace=ws(V=1 << 30)) == UNSUP
    grad = dict(h=at(1), W=at(2), tokens=at(3), lse=at(4), entropy=None, grad_logp=at(5),
                grad_entropy=None, dH=at(6), dW=at(7), status=None, H=8, V=100,
                dtype=torch.float32, workspace=Buf(8 << 58, 1 << 50))
    assert lp_bwd(**grad, N=65535 * 32) == OK
    assert lp_bwd(**grad, N=65535 * 32 + 1) == UNSUP


def test_cpu_tensors_are_refused():
    t, W = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8)
    for call in (lambda: m.flce_embedding(t, W), lambda: m.flce_rms_norm(W, torch.ones(8)),
                 lambda: m.flce_embedding_backward(t, torch.zeros(3, 8), 5),
                 lambda: m.flce_logprobs(torch.zeros(3, 8), W, t),
                 lambda: m.flce_rms_norm_backward(W, W, torch.ones(8), torch.ones(5))):
        with pytest.raises(ValueError, match="runs on a GPU"):
            call()
