"""Calls of the linear transform beside its usual ones: a slope asked for without an
activation, on each kernel that a size selects, and arguments whose square leaves
float32."""
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


def forward(x, w, activation, slope):
    """The C entry: the binding has no slope without an activation."""
    from lm_head_linear_amd import _lib
    (N, I), O = x.shape, w.shape[0]
    y = torch.empty(N, O, dtype=x.dtype, device=x.device)
    code = _lib.BF16 if x.dtype == torch.bfloat16 else _lib.F32
    rc = _lib.load().flce_linear(x.data_ptr(), I, w.data_ptr(), None, None, O, N, I, O,
                                 _lib.ACTIVATIONS[activation], y.data_ptr(), O, slope.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream, code, code)
    assert rc == _lib.OK
    return y


# up to 64 rows; a wide W; tiles of 128, 64 and (float32) 32, whole and partial; and from 192
# tiles of 256 (3592 x 3592: 225)
SIZES = [(1, 8, 24), (64, 64, 100), (65, 64, 100), (16, 64, 32768), (200, 136, 129), (512, 512, 512),
         (1900, 40, 2100), (6400, 64, 1024), (3592, 72, 3592)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,I,O", SIZES)
def test_slope_without_an_activation_is_one(N, I, O, dt):
    import lm_head_linear_amd as m
    g = torch.Generator(device="cuda").manual_seed(N)
    x, w, dy = (torch.randn(*s, generator=g, device="cuda").to(dt) for s in ((N, I), (O, I), (N, O)))
    sdt = torch.float16 if dt == torch.bfloat16 else dt
    slope = torch.full((N, O), float("nan"), device="cuda", dtype=sdt)
    y = forward(x, w, "none", slope)
    assert torch.equal(y, m.flce_linear(x, w)[0])
    assert bool((slope == 1).all())
    # the gradients are those of no slope: dz is dy
    for a, b in zip(m.flce_linear_backward(dy, x, w, slope), m.flce_linear_backward(dy, x, w)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [12, 300])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_arguments_of_any_finite_size(act, N, dt):
    """From 1e4 on every activation is z or zero and its slope one or zero in float32 (each
    factor's exponent is beyond 2^-149), up to the largest z, whose square is infinite."""
    import lm_head_linear_amd as m
    z = torch.tensor([1e4, 1e10, 1e18, 1.9e19, 1e25, 3e38], device="cuda")
    z = torch.cat([z, -z]).repeat((N + 11) // 12)[:N, None].to(dt)
    one = torch.ones(1, 1, device="cuda", dtype=dt)
    y, slope = m.flce_linear(z, one, activation=act, save_slope=True)
    assert torch.equal(y, torch.where(z > 0, z, torch.zeros_like(z)))
    assert torch.equal(slope, (z > 0).to(slope.dtype))
