"""The linear transform at sizes that take the head's 256 x 256 tiles (from 192 of them,
forward and backward apart), and those of 128 x 128 from odd rows and of float32: formulas in
float64 and tolerances of test_gpu_linear. Edges are no multiples of a tile, of a stage of k
or of each other."""
import pytest
import torch

from tests.test_gpu_linear import ACTS, U, check, half, inside, make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# tiles forward, backward: 289 and 297; 225 and 145 (the gradients on smaller ones); 153
# (smaller) and 225; 324 and 216, a k of whole stages, rows beyond a tile by one
BOTH, FWD, BWD, WHOLE = (4101, 2056, 4104), (3592, 1032, 3592), (4104, 2056, 2056), (4353, 1408, 4608)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lm_head_linear_amd._lib as L
    L.load()
    yield


@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("act", ACTS)
def test_both_ways(act, bias, residual):
    check(*BOTH, BF, act, bias, residual)


@pytest.mark.parametrize("size", [FWD, BWD, WHOLE])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_one_way_and_whole_stages(size, act):
    check(*size, BF, act, True, True)


@pytest.mark.parametrize("act", ACTS)
def test_float32_out_of_bf16_rows(act):
    check(*FWD, BF, act, act != "relu", act != "silu", ydt=torch.float32)


@pytest.mark.parametrize("ydt", [BF, torch.float32])
def test_strides_and_in_place(ydt):
    """Row strides and places that keep 16 bytes' alignment: the same tiles, the same bits;
    what lies between the rows stays. Others: the same sums to their error."""
    import lm_head_linear_amd as m
    N, I, O = FWD
    x, w, b, r, _ = make(N, I, O, BF, 1)
    want, slope = m.flce_linear(x, w, b, r, activation="silu", save_slope=True, y_dtype=ydt)
    xb, rb = torch.zeros(N, I + 24, device="cuda", dtype=BF), torch.zeros(N, O + 16, device="cuda", dtype=BF)
    xs, rs = xb[:, 8:8 + I], rb[:, 16:]
    xs.copy_(x)
    rs.copy_(r)
    yb = torch.full((N, O + 24), 7.0, device="cuda", dtype=ydt)
    y, s2 = m.flce_linear(xs, w, b, rs, activation="silu", save_slope=True, y=yb[:, 8:8 + O])
    assert torch.equal(y, want) and torch.equal(slope, s2)
    assert bool((yb[:, :8] == 7).all()) and bool((yb[:, 8 + O:] == 7).all())
    if ydt == BF:
        y, _ = m.flce_linear(xs, w, b, rs, activation="silu", y=rs)
        assert torch.equal(y, want) and y.data_ptr() == rs.data_ptr() and not rb[:, :16].any()
        return
    odd = torch.zeros(N, I + 3, device="cuda", dtype=BF)[:, 1:1 + I]
    odd.copy_(x)
    y, _ = m.flce_linear(odd, w, b, r, activation="silu", y_dtype=ydt)
    S = x.double().abs() @ w.double().abs().T + b.double().abs()
    inside(y, want.double(), 2 * 1.13 * 6 * (I + 1) ** 0.5 * U * S + 34 * U * (S + r.double().abs()).clamp_min(1), "y")


@pytest.mark.parametrize("size", [BOTH, BWD])
def test_accumulate_strides_and_parts(size):
    import lm_head_linear_amd as m
    N, I, O = size
    x, w, _, _, dy = make(N, I, O, BF, 3)
    slope = torch.rand(N, O, device="cuda").half()
    for s in (slope, None):                 # with a slope dz is dense, without it is dy's rows
        dx, dw, db = m.flce_linear_backward(dy, x, w, s)
        dyb, xb = (torch.full((N, n + 16), 7.0, device="cuda", dtype=BF) for n in (O, I))
        dyb[:, 8:8 + O], xb[:, 16:] = dy, x
        dxb = torch.full((N, I + 24), 7.0, device="cuda", dtype=BF)
        got = m.flce_linear_backward(dyb[:, 8:8 + O], xb[:, 16:], w, s, dx=dxb[:, 8:8 + I])
        assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db)))
        assert bool((dxb[:, :8] == 7).all()) and bool((dxb[:, 8 + I:] == 7).all())
        # added to: one rounding of the float32 sum, of which `new` was rounded once itself
        dw0, db0 = torch.randn(O, I, device="cuda").to(BF), torch.randn(O, device="cuda").to(BF)
        dx2, dw2, db2 = m.flce_linear_backward(dy, x, w, s, dweight=dw0.clone(), dbias=db0.clone(),
                                               accumulate=True)
        assert torch.equal(dx2, dx)
        for a, old, new in ((dw2, dw0, dw), (db2, db0, db)):
            want = old.double() + new.double()
            inside(a, want, half(BF) * (want.abs() + new.double().abs()) * 1.02
                   + U * (old.double().abs() + new.double().abs()), "added")
        # one alone runs on smaller tiles: the same sums to their error
        dz = dy.double() if s is None else (dy.float() * s.float()).to(BF).double()
        one, none, _ = m.flce_linear_backward(dy, x, w, s, want_dweight=False, bias=False)
        want = dz @ w.double()
        assert none is None
        inside(one, want, half(BF) * want.abs() * 1.02 + 6 * O ** 0.5 * U * (dz.abs() @ w.double().abs()), "dx")
        none, one, _ = m.flce_linear_backward(dy, x, w, s, want_dx=False, bias=False)
        want = dz.T @ x.double()
        assert none is None
        inside(one, want, half(BF) * want.abs() * 1.02 + 6 * N ** 0.5 * U * (dz.abs().T @ x.double().abs()), "dw")


def test_the_same_bits_again_and_nan_in_their_rows():
    import lm_head_linear_amd as m
    N, I, O = BOTH
    x, w, b, r, dy = make(N, I, O, BF, 9)
    y, s = m.flce_linear(x, w, b, r, activation="gelu_tanh", save_slope=True)
    g = m.flce_linear_backward(dy, x, w, s)
    for _ in range(2):
        y2, s2 = m.flce_linear(x, w, b, r, activation="gelu_tanh", save_slope=True)
        assert torch.equal(y, y2) and torch.equal(s, s2)
        assert all(torch.equal(p, q) for p, q in zip(g, m.flce_linear_backward(dy, x, w, s)))
    x[1, 3], x[N - 1, I - 1], dy[5, 7] = float("nan"), float("inf"), float("nan")
    y2, _ = m.flce_linear(x, w, b, r, activation="gelu_tanh")
    keep = torch.ones(N, dtype=torch.bool)
    keep[[1, N - 1]] = False
    assert torch.equal(y2[keep], y[keep]) and bool(y2[1].isnan().all())
    dx, dw, db = m.flce_linear_backward(dy, x, w, s)
    keep[:] = True
    keep[5] = False
    assert torch.equal(dx[keep], g[0][keep]) and bool(dx[5].isnan().all())
    assert bool(dw[7].isnan().all()) and bool(db[7].isnan()) and int(db.isnan().sum()) == 1


def test_captured():
    import lm_head_linear_amd as m
    x, w, b, r, dy = make(*BOTH, BF, 6)
    y, s = m.flce_linear(x, w, b, r, activation="silu", save_slope=True)
    want = [y, s, *m.flce_linear_backward(dy, x, w, s)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = m.flce_linear(x, w, b, r, activation="silu", save_slope=True)
        got = [y, s, *m.flce_linear_backward(dy, x, w, s)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        again = m.flce_linear_backward(dy, x, w, want[1])
        assert all(torch.equal(p, q) for p, q in zip(again, want[2:]))


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("N,I,O", [(2537, 1121, 3709), (2560, 1024, 3712)])
def test_tiles_of_128(N, I, O, dt):
    """580 of them forward; 441 and 392 for the gradients: odd rows and aligned ones."""
    for act, bias, residual in (("gelu", True, True), ("none", False, True)):
        check(N, I, O, dt, act, bias, residual)
