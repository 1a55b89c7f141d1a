"""How exact the heads' norm is in float32."""

import pytest
import torch

from matrix_optimizer_step_rot_gb300 import binding as B
from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    B.lib()


def roots(b, power, backward):
    """1 / sqrt of the mean square of heads (1, b) 2^power, 2^power times, as the kernels have it."""
    x = torch.stack([torch.ones_like(b), b], -1)[:, None] * 2.0 ** power
    w = torch.ones(2, device="cuda")
    if not backward:
        return ops.head_norm(x, w, eps=0.0)[0][:, 0, 0]
    # g = (-b, 1) has no part along x: dx = r g
    g = torch.stack([-b, torch.ones_like(b)], -1)[:, None]
    return ops.head_norm_backward(g, x, w, eps=0.0)[0][:, 0, 1] * 2.0 ** power


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("power", [-40, -1, 0, 30])
def test_root_of_a_row(power, backward):
    """Heads (1, b): with b of 11 bits their squares' mean is exact in float32, and an output is r itself (1 r 1;
    backward, with nothing along x, 1 1 r).  r is a Newton step from an approximation within 2^-22: what is left of
    that is 2^-43, and the last rounding is half a unit, at most E of r."""
    for b in (torch.arange(1, 1 << 11, device="cuda") * 2.0 ** -8, torch.arange(1, 1 << 11, device="cuda") * 2.0 ** -11):
        got = roots(b, power, backward).double()
        want = 1 / torch.sqrt((1 + b.double().square()) / 2)
        far = ((got - want).abs() / want).max().item()
        assert far <= E * (1 + 2.0 ** -18), far / E


@pytest.mark.parametrize("dim", [75, 128])
def test_error_is_no_more_than_that_of_rounded_steps(dim):
    """Over 2^14 heads: the error against that of the same formula by torch's correctly rounded root and quotient in
    float32.  Roundings are alike in number and size; a row's root is a sample of 2^14, so that two such errors agree
    to about 2^-7: 2% are allowed."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.randn(1 << 12, 4, dim, generator=g, device="cuda")
    dy = torch.randn(1 << 12, 4, dim, generator=g, device="cuda")
    w = 1 + 0.1 * torch.randn(dim, generator=g, device="cuda")

    def formula(x, dy, w):
        r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        hat, gw = x * r, dy * w
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w, \
            r * (gw - hat * (gw * hat).mean(-1, keepdim=True))

    want, plain = formula(x.double(), dy.double(), w.double()), formula(x, dy, w)
    got = ops.head_norm(x, w)[0], ops.head_norm_backward(dy, x, w)[0]
    for a, b, c in zip(got, plain, want):
        errors = [((t.double() - c).norm() / c.norm()).item() for t in (a, b)]
        assert errors[0] <= 1.02 * errors[1], errors


@pytest.mark.parametrize("dim", [1, 75, 128])
def test_rows_beyond_the_roots_range(dim):
    """Zeros, sums of squares beyond float32's range, an infinity: as the formula's float32 steps have it."""
    x = torch.ones(5, 1, dim, device="cuda")
    x[0], x[1], x[2, 0, 0], x[3, 0, dim - 1] = 0.0, 2.0 ** 70, float("inf"), float("nan")
    w = torch.ones(dim, device="cuda")
    for eps in (0.0, 1e-6):
        y = ops.head_norm(x, w, eps=eps)[0]
        want = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        near = (y - want).abs() <= 2.0 ** -20
        assert (near | torch.isnan(want)).all()
