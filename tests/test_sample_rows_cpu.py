"""Sampling from a head of few ids: the rows of a pass fit one grid (no GPU). A workgroup of
1024 threads takes a row, and a grid holds less than 2^32 threads."""
import os

import pytest
import torch

import lm_head_linear_amd as m
from lm_head_linear_amd import _lib

MOST = (2 ** 32 - 1) // 1024


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__ as g
        g.build()


@pytest.mark.parametrize("V", [1, 2, 7, 30, 31])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_of_a_pass(V, dt):
    """The workspace holds the logits of a pass: of MOST rows from there on."""
    size = lambda N: m.flce_sample_workspace_size(N, 8, V, dt)  # noqa: E731
    assert size(MOST) >= MOST * V * 4 and size(MOST - 1000) < size(MOST)
    assert size(MOST + 1) == size(1 << 23) == size((1 << 31) - 1) == size(MOST)


def test_logits_at_hand_are_one_pass():
    class At:
        def __init__(self, at, n=0):
            self.at, self.n = at, n

        def data_ptr(self):
            return self.at

        def numel(self):
            return self.n

        def element_size(self):
            return 1
    a = dict(logits=At(1 << 40), uniforms=At(1 << 42), V=1, tokens=At(1 << 44), workspace=At(1 << 46, 256))
    assert m.flce_sample_logits_check_args(N=MOST, **a) == _lib.OK
    assert m.flce_sample_logits_check_args(N=MOST + 1, **a) == _lib.ERR_UNSUPPORTED
