"""How exact the norm of the gradient is, and over which range.

A thread's at most 32 squares of a chunk are summed in float32 (a rounding each,
E = 2^-24 of the sum of positive terms), all beyond in float64; the root halves
that, and the result is rounded once: under 18 E whatever the number of elements.
The case past 2^31 elements tells such sums from float32 ones throughout: chains
of 2300 equal squares, as a thread would then have them, are off by 280 E."""

import pytest
import torch

from matrix_optimizer_step_rot_gb300 import binding as B
from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    B.lib()


def near(tensors):
    want = sum(t.double().square().sum().item() for t in tensors) ** 0.5
    got = ops.gradient_norm(tensors).item()
    assert abs(got - want) <= 18 * E * want, abs(got - want) / (E * want)


@pytest.mark.parametrize("sizes", [[1], [7, 0, 8192, 8193], [1 << 20, 3], [33] * 2500, [1 << 26]])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_error(sizes, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(sizes) % 1000)
    ts = [torch.randn(n, generator=g, device="cuda").to(dtype) for n in sizes]
    near(ts)
    near([torch.cat([t[:1], t])[1:] for t in ts])  # (off 16 bytes)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("value", [1 + 2.0 ** -12, 1.2345678, 1e-3])
def test_error_of_equal_numbers(value, shift):
    near([torch.full(((1 << 26) + shift,), value, device="cuda")[shift:]])


def test_past_2_31_elements():
    x = torch.full(((1 << 31) + 5000,), 1e-3, dtype=BF16, device="cuda")
    want = x[0].double().item() * x.numel() ** 0.5
    assert abs(ops.gradient_norm([x]).item() - want) <= 18 * E * want


def test_range():
    """A square within float32 counts as itself: to 2^64 above, to 2^-75 below (2^-150 is half its least number)."""
    def norm(*x):
        return ops.gradient_norm([torch.tensor(x, device="cuda")]).item()

    top = 2.0 ** 64 * (1 - E)  # its square rounds to float32's largest number
    assert norm(top) == pytest.approx(top, rel=2 * E) and norm(2.0 ** 64) == float("inf")
    assert norm(top, top) == pytest.approx(top * 2 ** 0.5, rel=2 * E)  # (of two threads: joined in float64)
    assert norm(2.0 ** -74) == 2.0 ** -74 and norm(2.0 ** -76) == 0.0 and norm(0.0) == 0.0
    assert norm(1.5 * 2.0 ** -75) == pytest.approx(2.0 ** -74.5, rel=2 * E)
    assert norm(2.0 ** -74, 1.0) == 1.0
