"""Tensors that a call writes in place: autograd notices that they are not what
its forward pass saw, as after torch's own in-place operations."""

import pytest
import torch

from matrix_optimizer_step_rot_gb300 import binding as B
from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops
from matrix_optimizer_step_rot_gb300.optimizer import AdamW, RotatedAdam

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    B.lib()


def normal(*shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(len(shape)), device="cuda")


@pytest.mark.parametrize("other", [False, True])
def test_a_parameter_stepped_between_forward_and_backward(other):
    stream = torch.cuda.Stream() if other else None
    w, x = normal(300).requires_grad_(), normal(300)
    opt = AdamW([w], lr=0.1)
    loss = (w * w * x).sum()
    if other:
        stream.wait_stream(torch.cuda.current_stream())
    opt.step([x], stream=stream)
    if other:
        torch.cuda.current_stream().wait_stream(stream)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    (w * w * x).sum().backward()
    assert torch.equal(w.grad, 2 * w.detach() * x)


def test_a_matrix_stepped_between_forward_and_backward():
    w, x = normal(64, 32).requires_grad_(), normal(64, 32)
    opt = RotatedAdam([(64, 32)], 1 << 20)
    loss = (w * w * x).sum()
    opt.step([w], [x], refresh=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("bits", [32, 8])
def test_what_adamw_writes(bits):
    p = [normal(300).bfloat16(), normal(70).half(), normal(5)]
    masters = [None, p[1].float(), None]
    states = [ops.adamw_state(t, bits=bits) for t in p]
    g = [t.float().clone() for t in p]
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    written, read = [*p, masters[1]], [*g, step]
    before = [t._version for t in written], [t._version for t in read]
    m, v = [s[0] for s in states], [s[1] for s in states]
    ops.adamw(p, g, m, v, step, lr=1e-3, masters=masters)
    assert [t._version for t in written] == [n + 1 for n in before[0]]
    assert [t._version for t in read] == before[1]
    with pytest.raises((ValueError, B.RotError)):  # (a refused call writes nothing)
        ops.adamw(p, g, m, v, 0, lr=1e-3, masters=masters)
    assert [t._version for t in written] == [n + 1 for n in before[0]]
    ops.adamw(p, g, m, v, step, lr=1e-3, masters=masters, counts=True)
    assert [t._version for t in written + read] == [n + 2 for n in before[0]] + before[1][:-1] + [before[1][-1] + 1]


def outputs():
    x, y = normal(40, 64), normal(40, 64)
    heads, keys, w = normal(9, 4, 64), normal(9, 2, 64), normal(64)
    rotary = ops.rotary_table(ops.rotary_frequencies(64))
    targets, one = torch.zeros(40, dtype=torch.int64, device="cuda"), torch.ones(40, device="cuda")
    a, b = (ops.fp8_quantize(t)[0] for t in (x, y))
    wt = ops.fp8_quantize(normal(32, 64), block_rows=128, transposed=True)[1]
    q, k = torch.empty_like(heads), torch.empty_like(keys)
    return {
        "dropout": ([torch.empty_like(x)], lambda o: ops.dropout(x, 0.5, 1, out=o)),
        "dropout_backward": ([torch.empty_like(x)], lambda o: ops.dropout_backward(x, 0.5, 1, out=o)),
        "policy_loss": ([x.clone()], lambda o: ops.policy_loss(o, targets, one, one, one, out=o)),
        "fp8_matmul": ([torch.zeros(40, 40, device="cuda")], lambda o: ops.fp8_matmul(a, b, out=o, accumulate=True)),
        "fp8_linear_backward": ([torch.empty(32, 64, device="cuda")],
                                lambda o: ops.fp8_linear_backward(normal(40, 32), x, wt, dw=o)),
        "rotate": ([q, k], lambda o, p: ops.rotate(heads, rotary, keys, out=o, k_out=p)),
        "rotate_backward": ([q, k], lambda o, p: ops.rotate_backward(heads, rotary, keys, out=o, k_out=p)),
        "head_norm": ([q, k], lambda o, p: ops.head_norm(heads, w, keys, w, out=o, k_out=p)),
        "head_norm_backward": ([q, k], lambda o, p: ops.head_norm_backward(heads, heads, w, keys, keys, w, out=o, k_out=p)),
    }


@pytest.mark.parametrize("name", ["dropout", "dropout_backward", "policy_loss", "fp8_matmul", "fp8_linear_backward",
                                  "rotate", "rotate_backward", "head_norm", "head_norm_backward"])
def test_outputs_that_are_given(name):
    given, call = outputs()[name]
    before = [t._version for t in given]
    call(*given)
    assert [t._version for t in given] == [n + 1 for n in before]


def test_inference_tensors_are_still_taken():
    with torch.inference_mode():
        x, p = normal(40, 64), normal(300)
        m, v = ops.adamw_state(p)
    ops.dropout(x, 0.5, 1, out=x)
    ops.adamw([p], [p.clone()], [m], [v], 1, lr=1e-3)
    assert torch.isfinite(p).all() and m.abs().max() > 0
