"""optimizer.AdamW and AdamW's lists without a GPU: what a refused call leaves
behind, what the object keeps of its parameters, how lists are read."""

import pytest
import torch

from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops
from matrix_optimizer_step_rot_gb300.optimizer import AdamW


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("norm", [None, torch.ones(())])
def test_a_refused_step_is_not_counted(captured, norm):
    w = torch.zeros(8)
    opt = AdamW([w], captured=captured)
    for grads in ([w], [], [None], 3):
        with pytest.raises(ValueError):
            opt.step(grads, norm=norm)
        assert int(opt.count) == 0


def test_the_device_count_is_refused_where_it_cannot_be():
    """Null and misaligned words; a step of the host."""
    import ctypes

    from matrix_optimizer_step_rot_gb300 import binding as B

    hyper = B.rot_adamw_hyper(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, scale=1.0, max_norm=1.0)
    call = B.lib().rot_adamw_step_counted
    good = 4096  # a stand-in: pointers are never followed on the way to a refusal
    for taken, work in ((0, good), (good + 4, good), (good, 0), (good, good + 8)):
        assert call(None, 0, ctypes.byref(hyper), taken, work, 0) == B.ROT_EINVAL
    assert call(None, 1, ctypes.byref(hyper), good, good, 0) == B.ROT_EINVAL
    assert call(None, 0, None, good, good, 0) == B.ROT_EINVAL
    if not torch.cuda.is_available():
        assert call(None, 0, ctypes.byref(hyper), good, good, 0) in (B.ROT_ECUDA, B.ROT_ENOTSUP)
    for step in (1, 3.0):
        with pytest.raises((ValueError, TypeError)):
            ops.adamw([], [], [], [], step, lr=0.1, counts=True)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_masters_keep_no_graph_of_their_parameters(dtype):
    """(A live graph of a leaf holds its gradient's node, and with it the stream that a captured backward pass would
    then have to use.)"""
    w = torch.randn(5, 7).to(dtype).requires_grad_()
    opt = AdamW([w], masters=True)
    master = opt.masters[0]
    assert not master.requires_grad and master.grad_fn is None and master.dtype == torch.float32
    assert torch.equal(master, w.detach().float()) and opt.params[0] is w
    assert not any(t.requires_grad for t in (opt.m[0], opt.v[0]))


def test_parameters_that_can_be_read_once_are_read_once():
    """Without masters: past the lists' lengths, so that what is refused is where the tensors are."""
    w = torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        ops.adamw(iter([w]), iter([w]), iter([w]), iter([w]), 1, lr=0.1)
    for masters in ([], [None, None], iter([])):
        with pytest.raises(ValueError, match="an entry for each parameter"):
            ops.adamw([w], [w], [w], [w], 1, lr=0.1, masters=masters)


def test_an_error_of_the_callers_generator_is_passed_on():
    def broken():
        yield torch.zeros(8)
        raise KeyError("the caller's own")

    w = torch.zeros(8)
    with pytest.raises(KeyError, match="the caller's own"):
        ops.gradient_norm(broken())
    with pytest.raises(KeyError, match="the caller's own"):
        ops.adamw([w], broken(), [w], [w], 1, lr=0.1)
    for bad in (3, None, object()):
        with pytest.raises(ValueError, match="expected a list"):
            ops.gradient_norm(bad)
