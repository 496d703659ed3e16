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
    (dict(workspace=None), WS), (dict(workspace=Buf(5 * M, 1024)), WS),
    (dict(workspace=Buf(5 * M + 128, 1 << 16)), WS),
])
def test_embedding_backward(kw, want):
    assert embed_bwd(**kw) == want


def test_embedding_workspace():
    size = m.flce_embedding_backward_workspace_size
    assert size(0, 8, 8) == 256 and size(1, 8, 0) == 0
    # one list of keys and positions, two partial rows for each 32 tokens
    assert size(16384, 4096, 131072) == 2 * 16384 * 4 + 2 * 512 * 4096 * 4
    # two lists beyond what one workgroup sorts, and 256 counts a block
    assert size(1 << 15, 64, 100) == 4 * (1 << 15) * 4 + 256 * 4 * 4 + 2 * 1024 * 64 * 4
    # windows grow with the tokens: the partial rows stay in proportion
    assert size(1 << 20, 64, 100) < 4 * (1 << 20) * 4 + 256 * 128 * 4 + 2 * 8192 * 64 * 4 + 1


def test_cpu_tensors_are_refused():
    t, W = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8)
    for call in (lambda: m.flce_embedding(t, W), lambda: m.flce_rms_norm(W, torch.ones(8)),
                 lambda: m.flce_embedding_backward(t, torch.zeros(3, 8), 5),
                 lambda: m.flce_rms_norm_backward(W, W, torch.ones(8), torch.ones(5))):
        with pytest.raises(ValueError, match="runs on a GPU"):
            call()
