"""optimizer.AdamW on the GPU: which steps it counts."""

import pytest
import torch

from matrix_optimizer_step_rot_gb300 import binding as B
from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops
from matrix_optimizer_step_rot_gb300.optimizer import AdamW

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    B.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def parameters(dtype=torch.float32):
    return [torch.randn(n, generator=gen(n), device="cuda").to(dtype) for n in (5000, 129)]


def gradients(k):
    return [torch.randn(n, generator=gen(1000 * k + n), device="cuda") * 1e-2 for n in (5000, 129)]


def word(x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


def contents(opt):
    return [t.clone() for t in opt.params] + [t for i in range(len(opt.params)) for t in opt.moments(i)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(contents(a), contents(b)))


@pytest.mark.parametrize("bits,dtype", [(32, torch.float32), (8, torch.bfloat16)])
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("skipped", [1, 3])
def test_steps_that_are_not_taken_are_not_counted(skipped, captured, bits, dtype):
    """An object that met norms that are not finite, before its first step and between two, equals one that did not."""
    a, b = (AdamW(parameters(dtype), lr=1e-2, weight_decay=0.1, bits=bits, captured=captured) for _ in range(2))
    for bad in [INF, NAN, -INF][:skipped]:
        a.step(gradients(9), norm=word(bad), max_norm=0.5)
    a.step(gradients(9), norm=word(1e30), scale=1e20)  # (their product is what is looked at)
    assert int(a.count) == 0 and same(a, b)
    for k in range(1, 4):
        norm = ops.gradient_norm(gradients(k))
        for opt in (a, b):
            opt.step(gradients(k), norm=norm, max_norm=0.5)
        a.step(gradients(8), norm=word(INF))
        assert int(a.count) == int(b.count) == k and same(a, b)
    assert all(not torch.equal(p, q) for p, q in zip(a.params, parameters(dtype)))


def test_replayed_steps_that_are_not_taken_are_not_counted():
    grads, norm = gradients(1), word(INF)
    a, b = (AdamW(parameters(), lr=torch.full((), 1e-2, device="cuda"), captured=True) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(grads, norm=norm, max_norm=0.5)
    for k, bad in enumerate((True, True, False, True, False, False)):
        for g, new in zip(grads, gradients(k + 2)):
            g.copy_(new)
        norm.copy_(word(NAN) if bad else ops.gradient_norm(grads))
        graph.replay()
        if not bad:
            b.step(grads, norm=norm, max_norm=0.5)
        assert torch.equal(a.count, b.count) and same(a, b)
    assert a.count.item() == 3


@pytest.mark.parametrize("other", [False, True])
def test_counted_on_the_host_then_on_the_device(other):
    """Steps without a norm, with one, without again: those of the operator at 1, 2, ..  A step counted on the device
    works its corrections out in float64 there, rounded once as on the host: at most a neighbouring number each, 4 E
    of the update, and a rounding each of two sums of about p."""
    stream = torch.cuda.Stream() if other else None
    opt, lr = AdamW(parameters(), lr=1e-2, weight_decay=0.1), 1e-2
    p = parameters()
    m, v = ([ops.adamw_state(t)[k] for t in p] for k in (0, 1))
    bound = [torch.zeros_like(t, dtype=torch.float64) for t in p]
    if other:
        stream.wait_stream(torch.cuda.current_stream())
    taken = 0
    for k, norm in enumerate((None, None, 1.0, INF, 1.0, None, NAN, None)):
        grads, at = gradients(k), None if norm is None else word(norm)
        if other:
            stream.wait_stream(torch.cuda.current_stream())
        opt.step(grads, norm=at, max_norm=2.0, stream=stream)
        if other:
            torch.cuda.current_stream().wait_stream(stream)
        if norm not in (INF, NAN):
            taken += 1
            before = [t.double() for t in p]
            ops.adamw(p, grads, m, v, taken, lr=lr, weight_decay=0.1)
            for i in range(2):
                u = (before[i] * (1 - lr * 0.1) - p[i].double()).abs()
                bound[i] += 4 * E * u + 2 * E * (before[i].abs() + p[i].double().abs())
        assert int(opt.count) == taken
        for i in range(2):
            assert torch.equal(opt.m[i], m[i]) and torch.equal(opt.v[i], v[i])
            assert ((opt.params[i].double() - p[i].double()).abs() <= bound[i]).all()


@pytest.mark.parametrize("captured", [False, True])
def test_a_refused_step_leaves_everything(captured):
    a, b = (AdamW(parameters(), lr=1e-2, captured=captured) for _ in range(2))
    norm = ops.gradient_norm(gradients(1))
    for grads, more in ((gradients(1)[:1], {}), ([None, None], {}), (gradients(1)[::-1], {}),
                        (gradients(1), dict(max_norm=0.0)), (gradients(1), dict(scale=NAN)),
                        (gradients(1), dict(norm=norm.cpu())), (gradients(1), dict(norm=norm.double()))):
        with pytest.raises((ValueError, B.RotError)):
            a.step(grads, **{"norm": norm, **more})
        assert int(a.count) == 0
    for opt in (a, b):
        opt.step(gradients(1), norm=norm)
    assert int(a.count) == 1 and same(a, b)


def test_a_training_step_captured_while_the_object_lives():
    """Forward and backward pass and the step in one graph, with masters of leaves that require gradients."""
    x = torch.randn(16, 32, generator=gen(1), device="cuda").half()
    first = torch.randn(32, generator=gen(2), device="cuda").half()
    w, u = (first.clone().requires_grad_() for _ in range(2))
    a, b = (AdamW([t], lr=1e-2, captured=True) for t in (w, u))

    def step(w, opt):
        (grad,) = torch.autograd.grad((x * w).float().square().mean(), w)
        opt.step([grad], norm=ops.gradient_norm([grad]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for opt, leaf in ((a, w), (b, u)):
            step(leaf, opt)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(w, a)
    for k in range(3):
        graph.replay()
        step(u, b)
    assert a.count.item() == 4 and torch.equal(w, u) and torch.equal(a.masters[0], b.masters[0])
    assert not torch.equal(w, first)


@pytest.mark.parametrize("other", [False, True])
def test_lists_that_can_be_read_once_without_masters(other):
    stream = torch.cuda.Stream() if other else None
    p, q, g = parameters(), parameters(), gradients(1)
    states = [[ops.adamw_state(t) for t in p] for _ in range(2)]
    ops.adamw(p, g, [s[0] for s in states[0]], [s[1] for s in states[0]], 1, lr=1e-2)
    if other:
        stream.wait_stream(torch.cuda.current_stream())
    ops.adamw(iter(q), iter(g), (s[0] for s in states[1]), (s[1] for s in states[1]), 1, lr=1e-2, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(p, q))
    assert all(torch.equal(a, b) for x, y in zip(*states) for a, b in zip(x, y))
