"""Outputs of the heads' operators that lie in memory which the same call reads
or writes otherwise are refused, before anything is done (without a GPU: past
this check, tensors of the host are refused for what they are)."""

import pytest
import torch

from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def calls(q, k, out, k_out, g=None, h=None):
    w, r = torch.ones(8), ops.Rotary(torch.zeros(4, dtype=torch.int64))
    g, h = (q, k) if g is None else (g, h)
    return [lambda: ops.rotate(q, r, k, out=out, k_out=k_out),
            lambda: ops.rotate_backward(q, r, k, out=out, k_out=k_out),
            lambda: ops.head_norm(q, w, k, w if k is not None else None, out=out, k_out=k_out),
            lambda: ops.head_norm_backward(q, g, w, k, h, w if k is not None else None, out=out, k_out=k_out)]


def new(heads=4):
    return torch.zeros(5, heads, 8)


def test_overlaps_are_refused():
    q, k, buffer = new(), new(), torch.zeros(7, 10, 8)
    part = torch.zeros(6, 4, 8)
    for given in ((q, k, k, None), (q, k, None, q), (q, k, k, q), (q, k, buffer[:5, :4], buffer[:5, :4]),
                  (q, q, q, None), (q, q, None, q), (q, k, (o := new()), o),
                  (part[:5], None, part[1:], None),  # a token further
                  (buffer[:5, :4], None, buffer.flatten()[:160].view(5, 4, 8), None),  # the same start, other rows
                  (q, part[:5], None, part[1:]), (q, part[:5], part[1:], None)):
        for call in calls(*given):
            with pytest.raises(ValueError, match="overlap"):
                call()
    g, h = new(), new()
    for out, k_out in ((h, None), (None, g)):  # the other side's forward inputs
        with pytest.raises(ValueError, match="overlap"):
            calls(q, k, out, k_out, g, h)[3]()


def test_what_is_allowed_comes_past_the_check():
    q, k, buffer = new(), new(2), torch.zeros(7, 10, 8)
    a, b = buffer[:5, :4], buffer[:5, 4:6]
    one = torch.zeros(1, 4, 8)
    for given in ((q, k, q, k), (q, k, None, None), (a, b, a, b), (q, k, new(), new(2)), (q, q, None, None), (q, None, q, None),
                  (one, None, one.as_strided((1, 4, 8), (99, 8, 1)), None), (q[:0], k[:0], q[:0], q[:0, :2])):
        for call in calls(*given):
            with pytest.raises(ValueError, match="CUDA"):
                call()
