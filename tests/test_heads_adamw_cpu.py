"""The heads' operators and AdamW without a GPU: what the entry points refuse,
calls with nothing to do, and the rotation's tables."""

import ctypes
import math

import numpy as np
import pytest
import torch

from matrix_optimizer_step_rot_gb300 import binding as B
from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops
from tests import heads_adamw_ref as ref

P = 4096  # a 256-byte aligned stand-in: pointers are never followed on the way to a refusal
F32, F16, BF16, E4M3 = B.ROT_TYPE_F32, B.ROT_TYPE_F16, B.ROT_TYPE_BF16, B.ROT_TYPE_E4M3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    B.lib()


def heads(n=4, data=P, batch=4096, token=256, head=32):
    return dict(data=data, heads=n, batch_stride=batch, token_stride=token, head_stride=head)


ROTARY = dict(turns=P, rotated=16, magnitude=1.0, interleaved=0, positions=P, position_bytes=8,
              position_batch_stride=5, position_token_stride=1, start=0)
CALLS = {
    "rot_rotate": dict(q=heads(), q_out=heads(), k=heads(2), k_out=heads(2), batch=2, tokens=5, dim=32, type=BF16,
                       rotary=ROTARY, inverse=0, stream=0),
    "rot_head_norm_forward": dict(q=heads(), q_weight=P, q_out=heads(), k=heads(2), k_weight=P, k_out=heads(2),
                                  wtype=F32, batch=2, tokens=5, dim=32, type=BF16, eps=1e-6, rotary=ROTARY, stream=0),
    "rot_head_norm_backward": dict(dq=heads(), q=heads(), q_weight=P, dq_out=heads(), dq_weight=P, dk=heads(2),
                                   k=heads(2), k_weight=P, dk_out=heads(2), dk_weight=P, wtype=F32, batch=2, tokens=5,
                                   dim=32, type=BF16, eps=1e-6, rotary=ROTARY, work=P, work_bytes=1 << 30, stream=0),
}


def run(name, **change):
    args = dict(CALLS[name], **change)
    assert set(change) <= set(CALLS[name])
    keep = []

    def arg(k, v):
        if not isinstance(v, dict):
            return None if v is None else v
        s = (B.rot_rotary if k == "rotary" else B.rot_heads)(**v)
        keep.append(s)
        return ctypes.byref(s)

    return getattr(B.lib(), name)(*[arg(k, v) for k, v in args.items()])


def rotary(**change):
    return dict(rotary=dict(ROTARY, **change))


SHARED = [dict(batch=-1), dict(tokens=-1), dict(batch=1 << 20, tokens=1 << 20), dict(dim=0), dict(dim=513),
          dict(type=E4M3), dict(type=-1), dict(q=None), dict(q=heads(-1)), dict(q=heads(65537)), dict(q=heads(data=0)),
          dict(q=heads(data=P + 1)), dict(q=heads(token=-1)), dict(q=heads(head=1 << 60)), dict(q=heads(3)),
          dict(k=heads(3)), dict(k=None), rotary(rotated=-2), rotary(rotated=17), rotary(rotated=34),
          rotary(turns=0), rotary(turns=P + 4), rotary(positions=P + 4), rotary(magnitude=NAN),
          rotary(positions=P + 2, position_bytes=4), rotary(position_bytes=2), rotary(position_token_stride=-1),
          rotary(position_batch_stride=-1)]
REFUSED = {
    "rot_rotate": SHARED + [dict(q_out=None), dict(q_out=heads(data=0)), dict(q_out=heads(head=31)),
                            dict(q_out=heads(token=127)), dict(q_out=heads(batch=0)), dict(q_out=heads(token=0)),
                            dict(q_out=heads(3)), dict(k_out=None), dict(k_out=heads(1)), dict(rotary=None)],
    "rot_head_norm_forward": SHARED + [dict(q_weight=0), dict(k_weight=0), dict(q_weight=P + 2), dict(k_weight=P + 1), dict(q_out=heads(head=16)), dict(q_out=None),
                                       dict(wtype=F16), dict(wtype=9), dict(eps=-1.0), dict(eps=NAN)],
    "rot_head_norm_backward": SHARED + [dict(dq=None), dict(dq=heads(3)), dict(dq=heads(data=P + 1)), dict(dk=None),
                                        dict(dk=heads(1)), dict(q_weight=0), dict(k_weight=0), dict(dq_weight=0),
                                        dict(dk_weight=0), dict(dq_weight=P + 2), dict(dk_weight=P + 1),
                                        dict(q_weight=P + 2), dict(dq_out=heads(head=16)), dict(wtype=F16),
                                        dict(eps=-1.0), dict(work=0), dict(work=P + 16), dict(work_bytes=1024),
                                        dict(k=None, dk=None, k_weight=0, dk_out=None)],
}


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in REFUSED.items() for c in cs])
def test_heads_refusals(name, change):
    assert run(name, **change) == B.ROT_EINVAL


@pytest.mark.parametrize("change", [
    dict(batch=0), dict(tokens=0), dict(q=heads(0), q_out=heads(0), k=heads(0), k_out=heads(0)),
    dict(tokens=0, q=heads(data=0), q_out=heads(data=0), k=heads(2, data=0), k_out=heads(2, data=0))])
def test_no_heads_need_no_device(change):
    assert run("rot_rotate", **change) == B.ROT_OK
    assert run("rot_head_norm_forward", **change) == B.ROT_OK


@pytest.mark.parametrize("name", sorted(CALLS))
def test_valid_heads_are_refused_for_want_of_a_gpu_alone(name):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    assert run(name) in (B.ROT_ECUDA, B.ROT_ENOTSUP)
    without = {k: None if k in ("k", "k_out", "dk", "dk_out") else 0
               for k in CALLS[name] if k in ("k", "k_out", "k_weight", "dk", "dk_out", "dk_weight")}
    assert run(name, **without) in (B.ROT_ECUDA, B.ROT_ENOTSUP)
    # heads before tokens, and inputs whose rows are one
    first = heads(4, token=32, head=160, batch=640)
    assert run(name, q=first, **{n: first for n in ("q_out", "dq_out") if n in CALLS[name]}) != B.ROT_EINVAL
    assert run(name, q=heads(4, token=0, head=0, batch=0)) != B.ROT_EINVAL


def test_head_norm_workspace():
    need = B.lib().rot_head_norm_work_bytes
    assert need(0) == 0 and need(513) == 0 and need(-1) == 0
    assert need(1) >= 8192 and need(512) == 8 * 512 * 1024


TENSOR = dict(p=P, g=P + 65536, m=P + 2 * 65536, v=P + 3 * 65536, m_scale=0, v_scale=0, master=0, n=1000, p_type=F32,
              g_type=BF16)
EIGHT = dict(m_scale=P + 4 * 65536, v_scale=P + 5 * 65536)
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, scale=1.0, max_norm=1.0, step=1, seed=3,
             lr_device=0, step_device=0, norm=P)


def adamw(*tensors, count=None, **hyper):
    arr = (B.rot_adamw_tensor * max(1, len(tensors)))(*[B.rot_adamw_tensor(**t) for t in tensors])
    h = B.rot_adamw_hyper(**dict(HYPER, **hyper))
    return B.lib().rot_adamw_step(arr, len(tensors) if count is None else count, ctypes.byref(h), 0)


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(n=(1 << 40) + 1), dict(p=0), dict(g=0), dict(m=0), dict(v=0), dict(p=P + 2), dict(g=P + 1),
    dict(m=P + 2), dict(v=P + 6), dict(p_type=E4M3), dict(g_type=7), dict(m_scale=P), dict(v_scale=P),
    dict(master=P + 6 * 65536), dict(p_type=F16), dict(p_type=F16, master=P + 2), dict(p_type=BF16, master=P + 2),
    dict(m=P), dict(v=P + 2 * 65536), dict(EIGHT, v_scale=P + 4 * 65536), dict(p_type=BF16, master=P)])
def test_adamw_tensor_refusals(change):
    assert adamw(dict(TENSOR, **change)) == B.ROT_EINVAL


@pytest.mark.parametrize("change", [
    dict(lr=-1.0), dict(lr=NAN), dict(eps=-1.0), dict(eps=NAN), dict(weight_decay=-1.0), dict(weight_decay=NAN),
    dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=NAN), dict(scale=NAN), dict(scale=INF), dict(step=0),
    dict(step=-3), dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=NAN), dict(count=-1),
    dict(norm=P + 2), dict(lr_device=P + 1), dict(step_device=P + 4)])
def test_adamw_hyper_refusals(change):
    assert adamw(TENSOR, **change) == B.ROT_EINVAL


def test_adamw_lists():
    assert adamw(TENSOR, TENSOR) == B.ROT_EINVAL  # the same arrays twice
    whole = dict(TENSOR, n=1 << 40)
    other = {k: v + (1 << 50) if k in ("p", "m", "v") else v for k, v in whole.items()}
    assert adamw(whole, other) == B.ROT_EINVAL  # 2^41 elements in all
    empty = dict(TENSOR, n=0, p=0, g=0, m=0, v=0)
    assert adamw() == B.ROT_OK and adamw(empty) == B.ROT_OK and adamw(empty, dict(empty, p_type=F16)) == B.ROT_OK
    assert B.lib().rot_adamw_step(None, 1, ctypes.byref(B.rot_adamw_hyper(**HYPER)), 0) == B.ROT_EINVAL
    assert B.lib().rot_adamw_step(None, 0, None, 0) == B.ROT_EINVAL
    if not torch.cuda.is_available():
        for t in (TENSOR, dict(TENSOR, p_type=BF16), dict(TENSOR, p_type=F16, master=P + 6 * 65536), dict(TENSOR, **EIGHT)):
            assert adamw(t, empty) in (B.ROT_ECUDA, B.ROT_ENOTSUP)
        assert adamw(TENSOR, step=0, step_device=P, norm=0, max_norm=0.0) in (B.ROT_ECUDA, B.ROT_ENOTSUP)


def norm(*tensors, count=None, out=P, work=P, work_bytes=1 << 20):
    arr = (B.rot_gradient * max(1, len(tensors)))(*[B.rot_gradient(*t) for t in tensors])
    return B.lib().rot_gradient_norm(arr, len(tensors) if count is None else count, out, work, work_bytes, 0)


def test_gradient_norm_refusals():
    good = (P, 100, F32)
    for call in (lambda: norm(good, count=-1), lambda: norm(good, out=0), lambda: norm(good, out=P + 2), lambda: norm(good, work=0),
                 lambda: norm(good, work=P + 16), lambda: norm(good, work_bytes=64), lambda: norm((0, 100, F32)),
                 lambda: norm((P + 2, 100, F32)), lambda: norm((P + 1, 100, BF16)), lambda: norm((P, -1, F32)),
                 lambda: norm((P, (1 << 40) + 1, F32)), lambda: norm((P, 1 << 40, F32), (P, 1, F32)),
                 lambda: norm((P, 100, E4M3))):
        assert call() == B.ROT_EINVAL
    need = B.lib().rot_gradient_norm_work_bytes
    assert need(-1) == 0 and need(0) == need(1000) == 8192 and need(1001) == 16384
    if not torch.cuda.is_available():
        assert norm(good, (0, 0, BF16)) in (B.ROT_ECUDA, B.ROT_ENOTSUP)


def test_python_refuses_what_is_not_on_the_gpu():
    x, w = torch.zeros(5, 4, 32), torch.ones(32)
    r = ops.rotary_table(ops.rotary_frequencies(32), device="cpu")
    for call in (lambda: ops.rotate(x, r), lambda: ops.rotate_backward(x, r), lambda: ops.rotate(None, r),
                 lambda: ops.head_norm(x, w), lambda: ops.head_norm_backward(x, x, w), lambda: ops.rotate(x, r.turns),
                 lambda: ops.adamw([w], [w], [w], [w], 1, lr=0.1), lambda: ops.adamw([None], [w], [w], [w], 1, lr=0.1),
                 lambda: ops.gradient_norm([w]), lambda: ops.gradient_norm([3])):
        with pytest.raises(ValueError):
            call()


def test_frequencies():
    f = ops.rotary_frequencies(8, 10000.0)
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.equal(ops.rotary_frequencies(8, factor=4.0), f / 4)
    assert ops.rotary_frequencies(0).numel() == 0
    # 2000 positions: 318, 32, 3.2 and 0.32 turns: kept, kept, 0.73 of the way, stretched
    g = ops.rotary_frequencies(8, factor=4.0, original_length=2000)
    blend = (2000 * 0.01 / (2 * math.pi) - 1) / 3
    want = torch.tensor([1.0, 0.1, 0.01 * (blend + (1 - blend) / 4), 0.001 / 4], dtype=torch.float64)
    assert torch.allclose(g, want, rtol=1e-12)
    # over the indices: the pair where the turns would be 2 lies halfway between those of 1 and 4
    h = ops.rotary_frequencies(8, factor=4.0, original_length=2 * 2 * math.pi / 0.01, by_index=True)
    assert h[2].item() == pytest.approx(0.01 * (0.5 + 0.5 / 4), rel=1e-12)
    for bad in (dict(rotated=7), dict(rotated=-2), dict(rotated=8, base=0.0), dict(rotated=8, factor=0.0),
                dict(rotated=8, original_length=10, low=2.0, high=1.0), dict(rotated=8, original_length=0)):
        with pytest.raises(ValueError):
            ops.rotary_frequencies(**bad)


def test_table():
    t = ops.rotary_table([2 * math.pi * 0.25, 2 * math.pi * 0.75, 2 * math.pi, 0.0, -2 * math.pi * 0.25], device="cpu")
    assert t.turns.tolist() == [1 << 62, -(1 << 62), 0, 0, -(1 << 62)]
    assert t.magnitude == 1.0 and not t.interleaved
    f = ops.rotary_frequencies(64)
    assert torch.equal(ops.rotary_table(f, device="cpu").turns,
                       torch.round(f / (2 * math.pi) * 2.0 ** 64).to(torch.int64))


def test_reference_rotation_of_a_worked_pair():
    """A quarter turn at position 1, half a turn at 2."""
    r = ops.Rotary(torch.tensor([1 << 62]), 2.0, False)
    x = torch.tensor([[[3.0, 4.0, 5.0]]]).expand(3, 1, 3)
    got = ref.rotated(x, r, torch.arange(3))
    want = torch.tensor([[6.0, 8.0, 5.0], [-8.0, 6.0, 5.0], [-6.0, -8.0, 5.0]], dtype=torch.float64)
    assert torch.allclose(got[:, 0], want, atol=1e-14)
    assert torch.allclose(ref.rotated(got, r, torch.arange(3), True)[..., :2], 4 * x[..., :2].double(), atol=1e-13)


def test_states_and_vectors():
    p = torch.zeros(5, 60)
    m, v = ops.adamw_state(p)
    assert m.shape == p.shape and v.dtype == torch.float32
    m, v = ops.adamw_state(p, bits=8)
    assert m.data.shape == p.shape and m.data.dtype == torch.float8_e4m3fn and v.scale.tolist() == [0, 0, 0]
    m.scale[1] = 130
    m.data.view(torch.uint8)[2, 8] = 0x38  # 1.0, element 128
    m.data.view(torch.uint8)[2, 7] = 0x38
    d = m.dequantize()
    assert d[2, 8].item() == 8.0 and d[2, 7].item() == 2.0 ** -127 and d.abs().sum().item() == pytest.approx(8.0)


def test_reference_grid():
    x = np.array([448.0, 17.0, 2.0 ** -6, 2.0 ** -9, 1e-5, 0.0])
    assert ref.scale_exponents(x).tolist() == [0.0] * 6 and ref.scale_exponents(x * 1.0001)[0] == 1.0
    assert ref.grid(x, np.zeros(6), 3, -6).tolist() == [32.0, 2.0] + [2.0 ** -9] * 4
