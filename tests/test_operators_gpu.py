"""The training operators on the GPU against plain 64-bit restatements
(tests/operators_ref.py), at the sizes, strides and values where they can go
wrong.

Tolerances.  u is the unit roundoff of an output's type (2^-24, 2^-11, 2^-8 for
float32, float16, bfloat16): one rounding of a result costs u |result|.
Float32 sums of n terms along a chain of c additions cost at most c 2^-24 times
the sum of the magnitudes; the chains are counted beside each test."""

import numpy as np
import pytest
import torch

from matrix_optimizer_step_rot_gb300 import binding as B
from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops
from tests import operators_ref as ref

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-44, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-39}
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    B.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows_of(g, rows, cols, pad, dtype, shift=0.0):
    """rows x cols of a buffer `pad` elements wider, the rest NaN."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda") + shift
    x[:, cols:] = float("nan")
    return x.to(dtype)[:, :cols]


def near(got, want, bound, what=""):
    """|got - want| <= bound element by element; NaN and infinities in the same places."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or over.max().item() <= 0, f"{what}: beyond its bound by {over.max().item():.3e}"


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

SEED, OFFSET = 0xFEDCBA9876543210, (7 << 33) + 5


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols,pad,p,with_res", [
    (1, 1, 0, 0.5, False), (1, 7, 0, 0.5, True), (3, 5, 2, 0.3, True), (257, 1001, 0, 0.25, False),
    (64, 128, 0, 0.1, True), (33, 136, 8, 0.1, True), (33, 136, 3, 0.1, True), (2, 4096, 0, 0.0, True),
    (5, 999, 0, 1.0, True), (1, 65537, 0, 0.5, False), (300, 4, 4, 0.7, False), (300, 2, 6, 0.7, True)])
def test_dropout(dtype, rows, cols, pad, p, with_res):
    g = gen(rows + cols)
    x = rows_of(g, rows, cols, pad, dtype)
    res = rows_of(g, rows, cols, 0, dtype) if with_res else None
    y = ops.dropout(x, p, SEED, OFFSET, residual=res)
    want = ref.dropped(x, p, SEED, OFFSET)
    # the product rounds once in float32, the sum once, the result once
    bound = U[dtype] * want.abs() + E * want.abs() + TINY[dtype]
    if with_res:
        total = want + res.double()
        bound = U[dtype] * total.abs() + E * (want.abs() + total.abs()) * 1.01 + TINY[dtype]
        want = total
    near(y, want, bound * 1.001)
    if not with_res:  # the mask itself, exactly
        assert torch.equal(y == 0, (want == 0) | (x == 0))


def test_dropout_ignores_what_it_drops():
    x = torch.full((64, 64), float("nan"), device="cuda")
    keep = torch.from_numpy(ref.kept(0, 4096, 0.5, 3, 0)).cuda().view(64, 64)
    y = ops.dropout(x, 0.5, 3, 0, residual=torch.ones(64, 64, device="cuda"))
    assert torch.equal(torch.isnan(y), keep) and torch.equal(y[~keep], torch.ones_like(y[~keep]))
    assert torch.equal(ops.dropout(x, 1.0, 3, 0), torch.zeros_like(x))


def test_dropout_mask_depends_on_seed_offset_and_position_alone():
    x = torch.ones(96, 40, device="cuda")
    a = ops.dropout(x, 0.5, 11, 4)
    wide = torch.ones(96, 43, device="cuda")[:, :40]
    assert torch.equal(a, ops.dropout(wide, 0.5, 11, 4))
    assert torch.equal(a, ops.dropout(x.view(2, 48, 40), 0.5, 11, 4).view(96, 40))
    assert torch.equal(a, ops.dropout(x.bfloat16(), 0.5, 11, 4).float())
    assert torch.equal(a, ops.dropout_backward(x, 0.5, 11, 4))
    assert not torch.equal(a, ops.dropout(x, 0.5, 12, 4))
    assert not torch.equal(a, ops.dropout(x, 0.5, 11, 5))
    y = x.clone()
    assert ops.dropout(y, 0.5, 11, 4, out=y) is y and torch.equal(a, y)


def test_dropout_rate():
    """2^24 elements: the share kept is within five standard deviations."""
    y = ops.dropout(torch.ones(1 << 24, device="cuda"), 0.1, 99, 0)
    share = (y != 0).double().mean().item()
    assert abs(share - 0.9) <= 5 * (0.1 * 0.9 / 2 ** 24) ** 0.5


def test_dropout_beyond_32_bit_counters():
    """Elements past 2^34 use the counter's upper word."""
    n = (1 << 34) + 40
    x = torch.ones(n, dtype=BF16, device="cuda")
    ops.dropout(x, 0.5, 21, 9, out=x)
    first = (1 << 34) - 32
    keep = torch.from_numpy(ref.kept(first, 72, 0.5, 21, 9)).cuda()
    assert torch.equal(x[first:] != 0, keep)
    assert torch.equal(x[:64] != 0, torch.from_numpy(ref.kept(0, 64, 0.5, 21, 9)).cuda())
    del x
    torch.cuda.empty_cache()


def test_dropout_on_another_stream():
    s = torch.cuda.Stream()
    x = torch.randn(1000, 77, device="cuda")
    want = ops.dropout(x, 0.3, 5, 6)
    s.wait_stream(torch.cuda.current_stream())
    y = ops.dropout(x, 0.3, 5, 6, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

NORM = [  # rows, cols, type, pad, residual, p, weight type, bias
    (1, 1, F32, 0, False, 0.0, F32, True),
    (1, 2048, BF16, 0, True, 0.0, F32, True),
    (5, 33, F32, 2, False, 0.1, F32, False),
    (9, 512, F16, 0, True, 0.1, F16, True),
    (7, 513, BF16, 0, True, 0.2, F32, True),
    (1000, 64, BF16, 8, False, 0.0, BF16, True),
    (333, 641, F32, 7, False, 0.0, F32, True),
    (3, 2049, F32, 0, True, 0.1, F32, True),
    (5, 4096, F16, 16, True, 0.1, F32, False),
    (3, 4097, BF16, 0, True, 0.0, BF16, True),
    (700, 2048, BF16, 0, True, 0.1, F32, True),
    (4, 8192, F32, 0, False, 0.0, F32, True),
    (3, 8200, BF16, 0, True, 0.1, F32, True),
    (3, 12289, F16, 0, True, 0.1, F32, True),
    (40, 12288, BF16, 0, True, 0.1, F32, True),
    (2, 16384, F32, 0, True, 0.1, F32, True),
    (2, 16385, BF16, 3, True, 0.1, F32, True),
    (1, 65536, F32, 0, False, 0.0, F32, True),
    # either side of the widths where the threads or the runs per row change
    (9, 256, BF16, 0, True, 0.1, F32, True), (9, 264, F16, 0, False, 0.1, F32, True),
    (6, 776, BF16, 0, True, 0.0, F32, True), (6, 1024, F16, 8, True, 0.1, F16, True),
    (6, 1032, BF16, 0, False, 0.0, F32, False), (5, 2056, BF16, 0, True, 0.1, F32, True),
    (3, 4104, F16, 0, True, 0.1, F32, True), (3, 5000, BF16, 0, False, 0.0, BF16, True),
    (3, 8193, BF16, 0, True, 0.1, F32, True), (2, 16392, F16, 0, True, 0.1, F32, True),
    (2, 20480, BF16, 0, True, 0.0, F32, True), (2, 32776, BF16, 0, True, 0.1, F32, True),
    (5, 128, F32, 0, True, 0.1, F32, True), (5, 516, F32, 4, True, 0.1, F32, True),
    (5, 1028, F32, 0, False, 0.1, F32, True), (3, 2052, F32, 0, True, 0.0, F32, False),
    (3, 6000, F32, 0, True, 0.1, F32, True), (2, 12000, F32, 0, True, 0.1, F32, True)]


def norm_inputs(rows, cols, dtype, pad, residual, wtype, bias, seed):
    g = gen(seed)
    x = rows_of(g, rows, cols, pad, dtype, shift=0.5)
    res = rows_of(g, rows, cols, 0, dtype) if residual else None
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(wtype)
    b = (0.2 * torch.randn(cols, generator=g, device="cuda")).to(wtype) if bias else None
    return x, res, w, b


def chain(cols):
    """Additions one after the other in a row's sum: at most 64 in a thread, 5
    in a warp, 32 over the warps; the mean's rounding and its use on top."""
    return 64 + 5 + 32 + 4


@pytest.mark.parametrize("rows,cols,dtype,pad,residual,p,wtype,bias", NORM)
def test_layer_norm(rows, cols, dtype, pad, residual, p, wtype, bias):
    x, res, w, b = norm_inputs(rows, cols, dtype, pad, residual, wtype, bias, rows + cols)
    y, h, mean, rstd = ops.layer_norm(x, w, b, 1e-5, residual=res, p=p, seed=SEED, offset=OFFSET)
    drop = ref.dropped(x, p, SEED, OFFSET)
    want = drop if res is None else drop + res.double()
    if res is None and p == 0:
        assert h is x
    else:
        near(h, want, (U[dtype] * want.abs() + 2 * E * (drop.abs() + want.abs())) * 1.01 + TINY[dtype], "h")
    y64, mean64, rstd64, hat = ref.norm(h, w, b, 1e-5)
    mag = h.double().abs().mean(1)
    dm = chain(cols) * E * mag  # the mean's error; half of it is also var's relative one
    near(mean, mean64, dm, "mean")
    rel = 2 * chain(cols) * E + 2 * (dm * rstd64)
    near(rstd, rstd64, rel * rstd64, "rstd")
    err = (dm * rstd64 + 2 * E * mag * rstd64)[:, None] + hat.abs() * (rel + 4 * E)[:, None]
    bound = err * w.double().abs() * 1.01 + 4 * E * y64.abs() + U[dtype] * y64.abs() * 1.01 + TINY[dtype]
    near(y, y64, bound, "y")


@pytest.mark.parametrize("rows,cols,dtype,pad,residual,p,wtype,bias", NORM)
def test_layer_norm_backward(rows, cols, dtype, pad, residual, p, wtype, bias):
    h, dh, w, _ = norm_inputs(rows, cols, dtype, pad, residual, wtype, bias, rows + 3 * cols)
    dy = rows_of(gen(7), rows, cols, 0, dtype)
    _, mean, rstd, _ = ref.norm(h, w, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    hat = (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    dx, dres, dw, db = ops.layer_norm_backward(dy, h, mean, rstd, w, dh=dh, p=p, seed=SEED,
                                               offset=OFFSET, bias=bias)
    g64, dw64, db64 = ref.norm_grad(dy, hat, rstd.double(), w, dh)
    wdy = (dy.double() * w.double()).abs()
    # hat rounds three times; each of the two means is a chain as above
    dhat = 3 * E * (hat.abs() + (h.double().abs() * rstd.double()[:, None]))
    s1, s2 = wdy.mean(1, keepdim=True), (wdy * hat.abs()).mean(1, keepdim=True)
    e1 = chain(cols) * E * s1
    e2 = chain(cols) * E * s2 + (wdy * dhat).mean(1, keepdim=True)
    err = rstd.double()[:, None] * (e1 + hat.abs() * e2 + dhat * s2 + 6 * E * (wdy + s1 + hat.abs() * s2))
    bound = err * 1.01 + (U[dtype] + 2 * E) * 1.01 * g64.abs() + TINY[dtype]
    if dh is not None:
        bound = bound + 2 * E * dh.double().abs()
    near(dres, g64, bound, "dresidual")
    if p == 0:
        assert dres is dx
    else:
        near(dx, ref.dropped(g64, p, SEED, OFFSET), 1.01 * ref.dropped(bound, p, SEED, OFFSET) + TINY[dtype]
             + 2 * U[dtype] * ref.dropped(g64, p, SEED, OFFSET).abs(), "dx")
    # a column's sum: a chain of rows per part, at most 608 parts in chains of 19, and the joins
    c = rows + 19 + 16
    near(dw, dw64, (c * E * (dy.double() * hat).abs().sum(0) + (dy.double().abs() * dhat).sum(0)) * 1.01 + 1e-37, "dweight")
    if bias:
        near(db, db64, c * E * dy.double().abs().sum(0) * 1.01 + 1e-37, "dbias")
    else:
        assert db is None


# Every plan of the norm: rows of single elements by their widths, then those of
# 16-byte runs; the last of each are too wide for the registers.  The rows are
# more than four times those that the blocks of the backward pass take at once
# (152 to 2432).
PLANS = [  # rows, cols, type, pad
    (9800, 77, BF16, 0), (9800, 128, F16, 1), (9800, 129, F32, 0), (9800, 199, BF16, 2), (9800, 256, BF16, 3),
    (4900, 257, F16, 0), (4900, 389, BF16, 0), (4900, 512, F32, 1), (2500, 513, BF16, 0), (2500, 777, F32, 0),
    (1300, 1025, BF16, 0), (2500, 1325, BF16, 0), (1300, 2047, F32, 2), (1300, 2049, F16, 0), (1300, 3001, BF16, 0),
    (650, 4097, F32, 0), (650, 6001, BF16, 0), (650, 8191, F16, 0), (270, 8195, BF16, 0),
    (9800, 264, BF16, 0), (9800, 512, F16, 8), (2500, 1040, BF16, 0), (2500, 516, F32, 0), (1300, 2056, BF16, 8),
    (1300, 1028, F32, 4), (650, 4104, F16, 0), (650, 2052, F32, 0), (650, 8200, BF16, 0), (650, 4100, F32, 0),
    (270, 16392, BF16, 0), (270, 8196, F32, 0)]


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("rows,cols,dtype,pad", PLANS)
def test_layer_norm_plans(rows, cols, dtype, pad, p):
    test_layer_norm(min(rows, 50), cols, dtype, pad, True, p, F32, True)
    test_layer_norm(min(rows, 50), cols, dtype, pad, False, p, dtype, False)


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("rows,cols,dtype,pad", PLANS)
def test_layer_norm_backward_plans(rows, cols, dtype, pad, p):
    """Rows as above.  The columns' sums: 8 rows of a block (or of a share of
    the columns' own kernel), 4 groups of it, 19 parts and 16 of the join, so
    that a row lost or taken twice is far beyond the bound."""
    test_layer_norm_backward(rows, cols, dtype, pad, True, p, F32, True)
    h, dh, w, _ = norm_inputs(rows, cols, dtype, pad, True, dtype, False, rows + cols)
    dy = rows_of(gen(7), rows, cols, 1, dtype)
    _, mean, rstd, _ = ref.norm(h, w, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    hat = (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for stream in (None, dh):
        _, _, dw, db = ops.layer_norm_backward(dy, h, mean, rstd, w, dh=stream, p=p, seed=SEED, offset=OFFSET)
        dhat = 3 * E * (hat.abs() + (h.double().abs() * rstd.double()[:, None]))
        sums = (dy.double() * hat).abs().sum(0)
        bound = (47 * E * sums + (dy.double().abs() * dhat).sum(0)) * 1.01
        assert bound.max().item() < 0.1  # (a row's share is of the order of 1)
        near(dw, (dy.double() * hat).sum(0), bound, "dweight")
        near(db, dy.double().sum(0), 47 * E * dy.double().abs().sum(0) * 1.01, "dbias")


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("rows,cols,dtype,pad", [
    (301, 200, BF16, 0), (301, 77, F32, 0), (301, 389, BF16, 0), (301, 1325, F16, 3), (301, 2048, BF16, 0),
    (161, 6001, BF16, 0), (161, 8200, F16, 0), (161, 8195, F32, 0), (70, 33000, BF16, 0)])
def test_layer_norm_in_its_inputs_place(rows, cols, dtype, pad, p):
    """The C entry points: the stream may take x's or the residual's place, the
    gradients that of the stream's gradient."""
    code = {F32: B.ROT_TYPE_F32, F16: B.ROT_TYPE_F16, BF16: B.ROT_TYPE_BF16}[dtype]
    lib, stream, ld = B.lib(), torch.cuda.current_stream().cuda_stream, cols + pad
    x, res, w, b = norm_inputs(rows, cols, dtype, pad, True, F32, True, 4)
    res = torch.empty(rows, ld, dtype=dtype, device="cuda")[:, :cols].copy_(res)
    y, h, mean, rstd = ops.layer_norm(x, w, b, residual=res, p=p, seed=SEED, offset=OFFSET)

    def copied(t):
        return torch.empty(rows, ld, dtype=dtype, device="cuda")[:, :cols].copy_(t)

    for own in (0, 1):
        given, y2 = [copied(x), copied(res)], torch.empty_like(y)
        mean2, rstd2 = torch.empty_like(mean), torch.empty_like(rstd)
        assert lib.rot_layer_norm_forward(
            given[0].data_ptr(), ld, given[1].data_ptr(), ld, w.data_ptr(), b.data_ptr(), B.ROT_TYPE_F32,
            given[own].data_ptr(), ld, y2.data_ptr(), cols, mean2.data_ptr(), rstd2.data_ptr(), rows, cols, code,
            1e-5, p, SEED, OFFSET, stream) == B.ROT_OK
        assert torch.equal(given[own], h) and torch.equal(given[1 - own], (res, x)[own])
        assert torch.equal(y2, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    dy, dh = copied(torch.randn(rows, cols, device="cuda")), copied(torch.randn(rows, cols, device="cuda"))
    dx, dres, dw, db = ops.layer_norm_backward(dy, h, mean, rstd, w, dh=dh, p=p, seed=SEED, offset=OFFSET)
    need = lib.rot_layer_norm_work_bytes(rows, cols)
    for own in (0, 1) if p > 0 else (0,):
        place, other = copied(dh), copied(torch.zeros(rows, cols, device="cuda"))
        outs = [place, other] if own == 0 else [other, place]
        work = torch.empty(need, dtype=torch.uint8, device="cuda")
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        assert lib.rot_layer_norm_backward(
            dy.data_ptr(), ld, h.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(), w.data_ptr(), B.ROT_TYPE_F32,
            place.data_ptr(), ld, outs[1].data_ptr() if p > 0 else None, ld, outs[0].data_ptr(), ld, dw2.data_ptr(),
            db2.data_ptr(), rows, cols, code, p, SEED, OFFSET, work.data_ptr(), need, stream) == B.ROT_OK
        assert torch.equal(outs[0], dx) and (p == 0 or torch.equal(outs[1], dres))
        assert torch.equal(dw2, dw) and torch.equal(db2, db)


def test_layer_norm_gradient_against_differences():
    """Directional derivatives of the forward kernel: central differences of
    sum(y r) in float32 with step 2^-6.  Rounding: outputs of magnitude <= 8
    carry 2^-21 each, 3000 of them at random add up to 55 2^-21 2.6e-5, over
    2 step: 8.4e-4.  Truncation: step^2 / 6 times the third derivative, at most
    a few times |v|^3 rstd^3 |r|: 4e-5 times a sum of 3000 random signs: 5e-3
    allowed."""
    rows, cols, step = 15, 200, 2.0 ** -6
    x, res, w, b = norm_inputs(rows, cols, F32, 0, True, F32, True, 5)
    g = gen(3)
    r = torch.randn(rows, cols, generator=g, device="cuda")
    kw = dict(p=0.2, seed=8, offset=2)

    def f(x, res, w, b):
        y = ops.layer_norm(x, w, b, 1e-5, residual=res, **kw)[0]
        return (y.double() * r.double()).sum().item()

    _, h, mean, rstd = ops.layer_norm(x, w, b, 1e-5, residual=res, **kw)
    dx, dres, dw, db = ops.layer_norm_backward(r, h, mean, rstd, w, **kw)
    args = [x, res, w, b]
    for i, grad in enumerate((dx, dres, dw, db)):
        v = torch.randn(args[i].shape, generator=g, device="cuda")
        v = v / v.norm()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * v, args[i] - step * v
        num = (f(*up) - f(*down)) / (2 * step)
        assert abs(num - (grad.double() * v.double()).sum().item()) <= 5e-3, i


def test_layer_norm_special_rows():
    """A constant row (variance 0), a row of zeros, and non-finite values that stay in their row."""
    x = torch.randn(6, 300, device="cuda")
    x[1] = 3.0
    x[2] = 0.0
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    w, b = torch.ones(300, device="cuda"), torch.full((300,), 0.25, device="cuda")
    y, _, mean, rstd = ops.layer_norm(x, w, b, 1e-5)
    assert torch.equal(y[2], b) and abs(rstd[2].item() - 1e-5 ** -0.5) < 1e-4
    assert (y[1] - 0.25).abs().max().item() <= 1e-6 * 1e-5 ** -0.5 * 3 * 2
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    assert torch.isfinite(y[[0, 1, 2, 5]]).all()


def test_layer_norm_of_no_rows():
    w = torch.ones(48, device="cuda")
    x = torch.empty(0, 48, device="cuda")
    y, h, mean, rstd = ops.layer_norm(x, w, w)
    assert y.shape == (0, 48) and mean.shape == (0,)
    dx, _, dw, db = ops.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, 48) and not dw.any() and not db.any()


def test_layer_norm_in_three_dimensions_and_twice_the_same():
    x = torch.randn(4, 50, 96, device="cuda", dtype=BF16)
    w = torch.randn(96, device="cuda")
    y, h, mean, rstd = ops.layer_norm(x, w, None, residual=x, p=0.1, seed=1)
    flat = ops.layer_norm(x.view(200, 96), w, None, residual=x.view(200, 96), p=0.1, seed=1)
    assert y.shape == x.shape and mean.shape == (4, 50)
    assert torch.equal(y.view(200, 96), flat[0]) and torch.equal(h.view(200, 96), flat[1])
    a = ops.layer_norm_backward(y, h, mean, rstd, w, p=0.1, seed=1)
    b = ops.layer_norm_backward(y, h, mean, rstd, w, p=0.1, seed=1)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_rows_of_more_dimensions_fold_where_they_can():
    """A slice of the last dimension of a 3-D tensor folds into rows; one of the
    middle dimension cannot."""
    full = torch.randn(4, 50, 96, device="cuda")
    w = torch.randn(64, device="cuda")
    part = full[:, :, :64]
    y = ops.layer_norm(part, w)[0]
    assert y.shape == (4, 50, 64) and torch.equal(y, ops.layer_norm(part.contiguous(), w)[0])
    assert torch.equal(ops.dropout(part, 0.4, 1), ops.dropout(part.contiguous(), 0.4, 1))
    one = full[:1, :1, :64].squeeze()  # a single row of one dimension
    assert torch.equal(ops.layer_norm(one, w)[0], y[0, 0]) and ops.layer_norm(one, w)[2].shape == ()
    with pytest.raises(ValueError):
        ops.dropout(full[:, :40], 0.4, 1)
    with pytest.raises(ValueError):
        ops.layer_norm(full.transpose(0, 2), torch.ones(4, device="cuda"))


# ---------------------------------------------------------------------------
# policy loss
# ---------------------------------------------------------------------------


def policy_inputs(tokens, vocab, dtype, pad, masked, seed):
    g = gen(seed)
    z = rows_of(g, tokens, vocab, pad, F32) * 2
    targets = torch.randint(vocab, (tokens,), generator=g, device="cuda")
    full = torch.empty(tokens, vocab + pad, dtype=dtype, device="cuda").fill_(float("nan"))
    full[:, :vocab] = z.to(dtype)
    z = full[:, :vocab]
    logp = torch.log_softmax(z.float(), 1).gather(1, targets[:, None])[:, 0]
    old = logp + 0.3 * torch.randn(tokens, generator=g, device="cuda")
    r = logp + 0.3 * torch.randn(tokens, generator=g, device="cuda")
    adv = torch.randn(tokens, generator=g, device="cuda")
    w = torch.rand(tokens, generator=g, device="cuda") + 0.5
    off = torch.rand(tokens, generator=g, device="cuda") < masked
    w[off], targets[off] = 0.0, -100
    for t in (old, r, adv):
        t[off] = float("nan")
    z[off] = float("nan")
    return z, targets, old, r, adv, w


def policy_bounds(z, targets, old, r, adv, w, lo, hi, kl):
    """(want, bounds of loss, logp, terms, gradient).  logp's error: the sum of
    exponentials is relative 2^-21 off (exponential 2 ulp, its argument rounded
    twice at magnitude <= 32, chains of additions between positive numbers),
    the logarithm and two subtractions round at its magnitude."""
    loss, logp, terms, grad = ref.policy(z, targets, old, r, adv, w, lo, hi, kl)
    on = w != 0
    # every exponential: argument error 2 * 32 * 2^-24 relative, 2 ulp; chain 300
    sum_rel = (64 + 4 + 300) * E
    dlp = torch.where(on, sum_rel + 4 * E * (logp.abs() + 32), 0.0)
    if old is None:
        return (loss, logp, terms, grad), dlp
    ratio = torch.where(on, torch.exp(logp - old.double()), 0.0)
    er = torch.where(on, torch.exp(r.double() - logp), 0.0) if r is not None else torch.zeros_like(ratio)
    # a term's slope in logp is |s| <= w (ratio |A| + kl (1 + exp(ref - logp))); its slope's slope the same size
    steep = torch.where(on, w.double() * (ratio * adv.double().abs() + kl * (1 + er)), 0.0)
    dterm = steep * (dlp + 16 * E) * 1.1 + 4 * E * terms.abs()
    s = steep * (dlp + 16 * E) * 1.1
    p = torch.where(on[:, None], torch.softmax(torch.where(on[:, None], z.double(), 0.0), 1), 0.0)
    onehot = torch.zeros_like(p).scatter_(1, targets.clamp(min=0)[:, None], 1.0)
    dgrad = s[:, None] * (p + onehot) + steep[:, None] * p * (sum_rel + 70 * E)
    return (loss, logp, terms, grad), dlp, dterm, dgrad


@pytest.mark.parametrize("tokens,vocab,dtype,pad,masked", [
    (1, 1, F32, 0, 0.0), (1, 131072, BF16, 0, 0.0), (3, 7, F32, 2, 0.3), (17, 257, F16, 0, 0.5),
    (64, 1024, BF16, 0, 0.2), (64, 1024, BF16, 8, 0.2), (9, 32768, F32, 0, 0.0), (5, 50021, BF16, 0, 0.2),
    (33, 4099, F32, 1, 0.2), (2, 151001, F32, 0, 0.0), (700, 600, F16, 0, 0.1), (4, 260000, F32, 0, 0.3)])
def test_policy_loss(tokens, vocab, dtype, pad, masked):
    z, targets, old, r, adv, w = policy_inputs(tokens, vocab, dtype, pad, masked, tokens + vocab)
    lo, hi, kl = 0.2, 0.3, 0.1
    f = np.float32
    (loss, logp, terms, grad), dlp, dterm, dgrad = policy_bounds(
        z, targets, old, r, adv, w, float(f(lo)), float(f(hi)), float(f(kl)))
    got = ops.policy_loss(z, targets, old, adv, w, ref_logp=r, clip_low=lo, clip_high=hi, kl_coef=kl)
    near(got[1], logp, dlp, "logp")
    # a ratio within rounding of a clip bound may fall on either side: those tokens' gradients are left out
    ratio = torch.exp(logp - old.double())
    edge = ((ratio - (1 - lo)).abs() < 1e-5) | ((ratio - (1 + hi)).abs() < 1e-5)
    near(got[2][~edge], grad[~edge], (dgrad + U[dtype] * grad.abs())[~edge] * 1.01 + TINY[dtype], "dlogits")
    assert abs(got[0].item() - loss.item()) <= dterm.sum().item() + E * abs(loss.item()) + 1e-30
    again = ops.policy_loss(z, targets, old, adv, w, ref_logp=r, clip_low=lo, clip_high=hi, kl_coef=kl)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    only = ops.policy_loss(z, targets, old, adv, w, ref_logp=r, clip_low=lo, clip_high=hi, kl_coef=kl, grad=False)
    assert only[2] is None and abs(only[0].item() - loss.item()) <= dterm.sum().item() + E * abs(loss.item()) + 1e-30
    near(ops.token_logprobs(z, targets, weights=w), logp, dlp, "token_logprobs")
    if masked == 0:
        near(ops.token_logprobs(z, targets), logp, dlp, "token_logprobs without weights")
    doubled = ops.policy_loss(z, targets, old, adv, w, ref_logp=r, clip_low=lo, clip_high=hi, kl_coef=kl,
                              grad_scale=4.0)[2]
    near(doubled[~edge], 4 * grad[~edge], 4 * (dgrad + U[dtype] * grad.abs())[~edge] * 1.01 + 4 * TINY[dtype], "scaled")


@pytest.mark.parametrize("tokens,vocab,dtype,pad,masked", [
    (1300, 325, BF16, 0, 0.2), (1300, 2047, F32, 1, 0.2), (2500, 4000, F16, 0, 0.1), (320, 5003, BF16, 5, 0.2),
    (310, 16384, F32, 0, 0.0), (400, 20000, BF16, 0, 0.2)])
def test_policy_loss_of_many_short_rows(tokens, vocab, dtype, pad, masked):
    """Rows of a warp, and of 128 threads."""
    test_policy_loss(tokens, vocab, dtype, pad, masked)


def from_largest(z):
    """The rows in 64 bits with their largest entry taken off: the same
    distribution, in numbers whose 64 bits are enough at any level."""
    z = z.double()
    return z - z.max(1, keepdim=True).values


def logp_bound(z, targets):
    """(log-probabilities in 64 bits, bound).  The numbers that count are the
    distances from the row's largest entry, e = (x - max) log2(e): each
    exponent rounds once (E |e|, and 3/4 more for the whole scale), an
    exponential is 2^-22 off, log2(e) as a float32 turns x - mean by E / 4; 40
    for the chains of additions and rescalings of at most 4 batches; the
    result and its two factors round at its size.  Nothing grows with the
    row's own level."""
    z = from_largest(z)
    full = z - torch.logsumexp(z, 1, keepdim=True)
    p = full.exp()
    e = z / np.log(2.0)
    e = torch.where(p > 0, e, 0.0)
    logp = full.gather(1, targets[:, None])[:, 0]
    mean = (p * torch.where(p > 0, full, 0.0)).sum(1)
    return logp, E * (44 + (p * (e.abs() + 1)).sum(1) + 3 * logp.abs() + 0.25 * (logp - mean).abs())


LEVELS = [0.0, 1e2, -1e2, 1e3, -1e3, 1e4, -1e4, 6e4, -6e4, 1e5, -1e5, 1e6, -1e6]


@pytest.mark.parametrize("dtype,level", [(t, x) for t in (F32, F16, BF16) for x in LEVELS
                                         if t != F16 or abs(x) < 65000])
def test_policy_loss_does_not_depend_on_the_rows_level(dtype, level):
    """Logits that lie together far from zero."""
    tokens, vocab = 48, 1000
    g = gen(int(abs(level)) + 1)
    z = (2 * torch.randn(tokens, vocab, generator=g, device="cuda", dtype=torch.float64) + level).to(dtype)
    targets = torch.randint(vocab, (tokens,), generator=g, device="cuda")
    logp, bound = logp_bound(z, targets)
    old = (logp + 0.3 * torch.randn(tokens, generator=g, device="cuda")).float()
    r = (logp + 0.3 * torch.randn(tokens, generator=g, device="cuda")).float()
    adv = torch.randn(tokens, generator=g, device="cuda")
    w = torch.rand(tokens, generator=g, device="cuda") + 0.5
    f = np.float32
    (loss, _, _, grad), _, dterm, dgrad = policy_bounds(z, targets, old, r, adv, w, float(f(0.2)), float(f(0.3)),
                                                        float(f(0.1)))
    got = ops.policy_loss(z, targets, old, adv, w, ref_logp=r, clip_low=0.2, clip_high=0.3, kl_coef=0.1)
    near(got[1], logp, bound, "logp")
    near(ops.token_logprobs(z, targets), logp, bound, "token_logprobs")
    ratio = torch.exp(logp - old.double())
    clear = ((ratio - 0.8).abs() > 1e-5) & ((ratio - 1.3).abs() > 1e-5)
    near(got[2][clear], grad[clear], (dgrad + U[dtype] * grad.abs())[clear] * 1.01 + TINY[dtype], "dlogits")
    assert abs(got[0].item() - loss.item()) <= dterm.sum().item() + E * abs(loss.item())


FAR = [-1e4, -6e4, -1e8, -1e9, -1.5e9, -1e10, -1e12, -1e15, -1e30, 1e4, 1e8, 1e9, 1e10, 1e12, 1e15, 1e30]


@pytest.mark.parametrize("dtype,level", [(t, x) for t in (F32, F16, BF16) for x in FAR if t != F16 or abs(x) < 65000])
def test_policy_loss_far_from_zero(dtype, level):
    """Whole rows of one number, rows next to it (spacings of the type at that
    level apart), and rows of which a part is that number."""
    g = gen(5)
    vocab = 40
    z = torch.full((12, vocab), level, device="cuda", dtype=torch.float64)
    step = abs(level) * 2 * U[dtype]  # (about a spacing)
    z[4:8] += step * torch.randint(-2, 3, (4, vocab), generator=g, device="cuda")
    z[8:, 5:] = torch.randn(4, vocab - 5, generator=g, device="cuda").double()
    z = z.to(dtype)
    targets = torch.randint(vocab, (12,), generator=g, device="cuda")
    targets[8:] = z[8:].argmax(1)
    logp, bound = logp_bound(z, targets)
    one = torch.ones(12, device="cuda")
    old, ref_ = (logp - 0.1).float(), (logp + 0.05).float()
    f = np.float32
    # (a logp far below -100 rounds by more than a ratio could be told from)
    w = torch.where(logp > -100, one, 0.0)
    (loss, _, _, grad), _, dterm, dgrad = policy_bounds(from_largest(z), targets, old, ref_, one, w, float(f(0.2)),
                                                        float(f(0.2)), float(f(0.1)))
    near(ops.token_logprobs(z, targets), logp, bound, "token_logprobs")
    got = ops.policy_loss(z, targets, old, one, w, ref_logp=ref_, kl_coef=0.1)
    on = w != 0
    near(got[1][on], logp[on], bound[on], "logp")
    near(got[2], grad, (dgrad + U[dtype] * grad.abs()) * 1.01 + TINY[dtype], "dlogits")
    assert abs(got[0].item() - loss.item()) <= dterm.sum().item() + E * abs(loss.item())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_policy_loss_of_targets_at_the_lowest_value(dtype):
    """A target masked with the type's lowest value has a finite
    log-probability: its distance from the rest."""
    lowest = torch.finfo(dtype).min
    z = torch.randn(6, 300, generator=gen(8), device="cuda").to(dtype)
    targets = torch.arange(6, device="cuda") * 50
    z[torch.arange(6), targets] = lowest
    logp, bound = logp_bound(z, targets)
    assert torch.isfinite(logp).all()
    got = ops.token_logprobs(z, targets)
    near(got, logp, bound, "logp")
    one = torch.ones(6, device="cuda")
    loss, _, d = ops.policy_loss(z, targets, got, one, one / 6, ref_logp=got, kl_coef=0.1)
    assert torch.isfinite(d).all()
    if dtype == F16:  # (the ratio to the rounded log-probability: within 2^-9 of 1)
        assert abs(loss.item() + 1) <= 2.0 ** -8
    else:
        assert abs(loss.item() + 1) <= 8 * E


def test_policy_loss_without_weight_on_the_penalty():
    """kl_coef 0: a reference far above the policy is not part of the loss."""
    z, targets, old, r, adv, w = policy_inputs(40, 1000, BF16, 0, 0.3, 1)
    want = ops.policy_loss(z, targets, old, adv, w)
    got = ops.policy_loss(z, targets, old, adv, w, ref_logp=old + 200.0)
    assert torch.isfinite(want[0]) and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("delta", [0.0, 1e-6, 1e-5, 1e-4, 1e-3, 1e-2, 0.1, 0.24, 0.3, 0.49, 0.51, 1.0, 3.0])
def test_policy_penalty_near_the_reference(delta):
    """The penalty alone (advantages 0, ratio 1): exp(r) - r - 1 with r = ref -
    logp, relative to itself.  Rows of two equal logits, whose logp of -log 2
    the kernel holds to 48 bits: r rounds twice at most (E each, twice that in
    the term), the series and its two products 3 E; from 1/2 on the
    exponential's last place and the difference, 4 E of the term.  At delta 0,
    r is what float32 leaves of log 2, good to E^2."""
    z = torch.zeros(64, 2, device="cuda")
    targets = torch.zeros(64, dtype=torch.int64, device="cuda")
    sign = torch.where(torch.arange(64, device="cuda") % 2 == 0, 1.0, -1.0)
    ref_ = (-np.log(2.0) + delta * sign.double()).float()
    logp = torch.full((64,), -np.log(2.0), device="cuda", dtype=torch.float64)
    r = ref_.double() - logp
    zero, one = torch.zeros(64, device="cuda"), torch.ones(64, device="cuda")
    want = torch.where(r.abs() < 0.02, r * r * (0.5 + r / 6 + r * r / 24 + r ** 3 / 120), torch.expm1(r) - r)
    # (below 0.02 the series' next term is r^4 / 360 of it: 5e-10)
    for i in (0, 1):
        loss, _, _ = ops.policy_loss(z[i:i + 1], targets[:1], logp[:1].float(), zero[:1], one[:1],
                                     ref_logp=ref_[i:i + 1], kl_coef=1.0, grad=False)
        w, ri = want[i].item(), abs(r[i].item())
        assert abs(loss.item() - w) <= 8 * E * w + 1.2 * (ri + ri * ri) * 8 * E * E + 64 * E ** 4, (loss.item(), w)


def test_policy_loss_of_no_advantage_is_the_penalty_alone():
    """Advantage 0 under a ratio beyond float32: 0, not 0 times infinity."""
    z, targets, old, r, adv, w = policy_inputs(40, 1000, F32, 0, 0.3, 1)
    adv = torch.where(w != 0, 0.0, adv)
    want = ops.policy_loss(z, targets, old, adv, w, ref_logp=r, kl_coef=0.1)
    got = ops.policy_loss(z, targets, old - 200.0, adv, w, ref_logp=r, kl_coef=0.1)
    assert torch.isfinite(want[0]) and all(torch.equal(a, b) for a, b in zip(want, got))


def test_policy_loss_in_place_and_without_reference():
    z, targets, old, _, adv, w = policy_inputs(40, 1000, BF16, 0, 0.3, 1)
    want = ops.policy_loss(z, targets, old, adv, w)
    own = z.clone()
    got = ops.policy_loss(own, targets, old, adv, w, out=own)
    assert got[2] is own and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("tokens,vocab,dtype,pad", [
    (1300, 325, BF16, 0), (1300, 1024, BF16, 0), (1400, 1999, F32, 1), (1300, 4000, F16, 0), (400, 20000, BF16, 0),
    (5, 70001, F32, 0)])
def test_policy_gradient_in_the_logits_place(tokens, vocab, dtype, pad):
    """One plan after the other (a warp, 128 or 512 threads, a cluster): the same bits as in a new tensor."""
    z, targets, old, r, adv, w = policy_inputs(tokens, vocab, dtype, pad, 0.2, 3)
    want = ops.policy_loss(z, targets, old, adv, w, ref_logp=r, kl_coef=0.1)
    own = torch.empty(tokens, vocab + pad, device="cuda", dtype=dtype)[:, :vocab].copy_(z)
    got = ops.policy_loss(own, targets, old, adv, w, ref_logp=r, kl_coef=0.1, out=own)
    assert got[2] is own and all(torch.equal(a, b) for a, b in zip(want, got))


def test_policy_loss_special_rows():
    """Masked vocabulary entries (-inf), the type's lowest value, an empty
    distribution, targets outside the vocabulary, infinite logits: as the
    formula has it, each in its own row."""
    lowest = torch.finfo(F32).min
    z = torch.zeros(8, 40, device="cuda")
    z[0, 5:] = float("-inf")
    z[1, 5:] = lowest
    z[2] = float("-inf")
    z[3, 3] = float("inf")
    z[4, 3] = float("nan")
    z[5, :35] = float("-inf")
    z[7] = lowest
    targets = torch.tensor([2, 2, 2, 2, 2, 39, 40, 1], device="cuda")
    one = torch.ones(8, device="cuda")
    loss, logp, d = ops.policy_loss(z, targets, -one, one, one, ref_logp=-one, kl_coef=0.1)
    nan = torch.tensor([False, False, True, True, True, False, True, False], device="cuda")
    assert torch.equal(torch.isnan(logp), nan) and torch.isnan(loss)
    assert torch.isnan(d[nan]).all() and torch.isfinite(d[~nan]).all()
    five = float(np.log(5.0))
    assert (logp[[0, 1, 5]] + five).abs().max().item() <= 4 * E * five + 8 * E
    assert abs(logp[7].item() + np.log(40.0)) <= 16 * E
    assert not d[0, 5:].any() and not d[1, 5:].any() and not d[5, :35].any()
    keep = torch.where(nan, 0.0, one)
    loss, logp, d = ops.policy_loss(z, targets, -one, one, keep, ref_logp=-one, kl_coef=0.1)
    assert torch.isfinite(loss) and not d[nan].any() and not logp[nan].any()


def test_policy_gradient_against_differences():
    """d(loss) along random directions, float32 logits, unclipped tokens only
    (ratio 1, 20% from a bound): step 2^-7 over vectors of length 1.  Rounding:
    a loss near 1 carries 2^-22, over 2 step: 1.5e-5; truncation step^2 / 6
    times a third derivative below 8: 8e-5."""
    z, targets, old, r, adv, w = policy_inputs(6, 50, F32, 0, 0.0, 4)
    old = ops.token_logprobs(z, targets)
    w = w / w.sum()
    kw = dict(ref_logp=r, kl_coef=0.5)
    d = ops.policy_loss(z, targets, old, adv, w, **kw)[2]
    for seed in range(4):
        v = torch.randn(z.shape, generator=gen(seed), device="cuda")
        v, step = v / v.norm(), 2.0 ** -7
        up = ops.policy_loss(z + step * v, targets, old, adv, w, grad=False, **kw)[0].item()
        down = ops.policy_loss(z - step * v, targets, old, adv, w, grad=False, **kw)[0].item()
        assert abs((up - down) / (2 * step) - (d.double() * v.double()).sum().item()) <= 1.5e-4


def test_policy_loss_of_no_tokens():
    z = torch.empty(0, 16, device="cuda")
    e = torch.empty(0, device="cuda")
    loss, logp, d = ops.policy_loss(z, e.long(), e, e, e)
    assert loss.item() == 0 and logp.shape == (0,) and d.shape == (0, 16)


def test_policy_loss_past_2_31_logits():
    """20000 x 131072 bfloat16 logits (2.6e9): the last rows, by themselves."""
    tokens, vocab = 20000, 131072
    z = torch.zeros(tokens, vocab, dtype=BF16, device="cuda")
    z[-2:] = torch.randn(2, vocab, generator=gen(2), device="cuda").to(BF16)
    targets = torch.full((tokens,), vocab - 1, device="cuda")
    one = torch.ones(tokens, device="cuda")
    old, w = -11.5 * one, one / tokens
    _, logp, d = ops.policy_loss(z, targets, old, one, w, out=None)
    tail = ops.policy_loss(z[-2:], targets[-2:], old[-2:], one[-2:], w[-2:])
    # two sums of the same row, each within 400 2^-24 of it (policy_bounds), and their roundings
    near(logp[-2:], tail[1], torch.full((2,), 1000 * E, device="cuda"))
    near(d[-2:], tail[2], (2 * U[BF16] + 1000 * E) * tail[2].double().abs() * 1.01 + TINY[BF16])
    assert abs(logp[0].item() + np.log(vocab)) <= 1e-5
    del z, d
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# 8-bit matrices
# ---------------------------------------------------------------------------


def spread(g, rows, cols, dtype):
    """Values over many magnitudes, so that blocks differ in scale."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-10, 4, (rows, 1), generator=g, device="cuda").float())
    return x.to(dtype)


def check_quantized(m, x, block_rows, dtype):
    q, scale = ref.quantize(x.double().cpu().numpy(), block_rows, dtype)
    assert np.array_equal(m.scale.cpu().numpy(), scale)
    got = m.data.float().double().cpu().numpy()
    assert np.array_equal(got, q, equal_nan=True)


@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("rows,cols,dtype,block_rows,pad", [
    (1, 1, F32, 1, 0), (3, 130, BF16, 1, 0), (128, 128, F16, 128, 0), (129, 257, F32, 128, 0), (200, 384, BF16, 1, 8),
    (65, 127, F16, 1, 1), (300, 136, F32, 128, 4), (1, 2048, BF16, 1, 0), (257, 16, BF16, 128, 0)])
def test_quantize(fmt, rows, cols, dtype, block_rows, pad):
    x = spread(gen(rows + cols), rows, cols + pad, dtype)[:, :cols]
    q, t = ops.fp8_quantize(x, block_rows=block_rows, transposed=True, dtype=fmt)
    check_quantized(q, x, block_rows, fmt)
    check_quantized(t, x.t(), block_rows, fmt)
    only, none = ops.fp8_quantize(x, block_rows=block_rows, dtype=fmt)
    assert none is None and torch.equal(only.data.view(torch.uint8), q.data.view(torch.uint8))
    none, only = ops.fp8_quantize(x, block_rows=block_rows, rows=False, transposed=True, dtype=fmt)
    assert none is None and torch.equal(only.data.view(torch.uint8), t.data.view(torch.uint8))


@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_values(fmt, block_rows):
    """Blocks of zeros, subnormal and largest floats, values on and beside the
    scales' steps, NaN and infinities in their own places."""
    x = torch.randn(256, 256, generator=gen(1), device="cuda")
    x[:128, :128] = 0.0
    x[:128, 128:] *= 1e-42
    x[130, 3], x[131, 200], x[132, 7] = float("nan"), float("inf"), float("-inf")
    x[140, :] = 448.0
    x[141, :] = float(np.nextafter(np.float32(448), np.float32(1e9)))
    x[142, :] = 57344.0
    x[143, :] = 3.4028234663852886e38
    x[144, :] = -0.0
    q, t = ops.fp8_quantize(x, block_rows=block_rows, transposed=True, dtype=fmt)
    check_quantized(q, x, block_rows, fmt)
    check_quantized(t, x.t(), block_rows, fmt)


PRODUCT = [(1, 1, 1), (1, 6144, 2048), (3, 130, 16), (128, 128, 128), (127, 129, 131), (200, 300, 4096), (64, 2048, 500),
           (513, 40, 1030), (16, 16, 20000), (1, 128, 70000), (300, 520, 129), (40, 1000, 640), (129, 193, 513),
           (256, 384, 1024), (9, 192, 512), (1000, 385, 4100), (3000, 2000, 130)]


def product_bound(a, b, K):
    """Each stretch of K is summed on the tensor cores, whose additions may
    truncate (2^-23) and align up to 32 products at a time; stretches join in
    float32."""
    mag = a.abs() @ b.abs().t()
    return (64 + K / 512) * 2 * E * mag


@pytest.mark.parametrize("M,N,K", PRODUCT)
@pytest.mark.parametrize("ra,rb,fa,fb", [(1, 128, E4, E4), (1, 1, E5, E4), (128, 128, E4, E5), (128, 1, E5, E5)])
def test_product(M, N, K, ra, rb, fa, fb):
    g = gen(M + N + K)
    a = ops.fp8_quantize(spread(g, M, K, F32), block_rows=ra, dtype=fa)[0]
    b = ops.fp8_quantize(spread(g, N, K, F32), block_rows=rb, dtype=fb)[0]
    va, vb = ref.values(a), ref.values(b)
    want, bound = va @ vb.t(), product_bound(va, vb, K)
    got = ops.fp8_matmul(a, b)
    near(got, want, bound, "float32")
    assert torch.equal(got, ops.fp8_matmul(a, b))
    if ra == 1 and rb == 128:
        for dtype in (F16, BF16):
            small = want.abs() <= 6e4
            near(torch.where(small, ops.fp8_matmul(a, b, dtype=dtype).double(), 0.0), torch.where(small, want, 0.0),
                 bound + (want.abs() + bound) * U[dtype] * 1.01 + TINY[dtype], str(dtype))
        c = torch.randn(M, N + 3, generator=g, device="cuda")
        before = c.clone()
        out = c[:, :N]
        ops.fp8_matmul(a, b, out=out, accumulate=True)
        near(out, before[:, :N].double() + want, bound + 2 * E * (want.abs() + before[:, :N].abs()), "accumulated")
        assert torch.equal(c[:, N:], before[:, N:])
    assert ops.status() == B.ROT_OK


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 1), (37, 2048), (700, 513), (6144, 640), (5, 12288)])
def test_product_of_few_rows(M, N, K):
    """Either side of the row count where another kernel takes over; a layer's
    own rounding of x gives what fp8_quantize gives."""
    g = gen(M + N + K)
    x = spread(g, M, K, BF16)
    a = ops.fp8_quantize(x)[0]
    b = ops.fp8_quantize(spread(g, N, K, F32), block_rows=128)[0]
    va, vb = ref.values(a), ref.values(b)
    want, bound = va @ vb.t(), product_bound(va, vb, K)
    near(ops.fp8_matmul(a, b), want, bound, "8-bit rows")
    y = ops.fp8_linear(x, b)
    near(y, want, bound + (want.abs() + bound) * U[BF16] * 1.01 + TINY[BF16], "layer")
    c = torch.ones(M, N, device="cuda")
    ops.fp8_matmul(a, b, out=c, accumulate=True)
    near(c, 1 + want, bound + 2 * E * (want.abs() + 1), "accumulated")


@pytest.mark.parametrize("N", [300, 301, 571])
def test_product_whose_cut_columns_come_again(N):
    """Several tiles to an SM, of which every other one is cut within the
    columns that a warp stores at once."""
    g = gen(N)
    M, K = 128 * 308 + 5, 130
    a = ops.fp8_quantize(torch.randn(M, K, generator=g, device="cuda"))[0]
    b = ops.fp8_quantize(torch.randn(N, K, generator=g, device="cuda"), block_rows=128)[0]
    va, vb = ref.values(a), ref.values(b)
    want, bound = va @ vb.t(), product_bound(va, vb, K)
    near(ops.fp8_matmul(a, b), want, bound, "float32")
    near(ops.fp8_matmul(a, b, dtype=BF16), want, bound + (want.abs() + bound) * U[BF16] * 1.01 + TINY[BF16], "bfloat16")
    c = torch.ones(M, N, device="cuda")
    ops.fp8_matmul(a, b, out=c, accumulate=True)
    near(c, 1 + want, bound + 2 * E * (want.abs() + 1), "accumulated")
    assert ops.status() == B.ROT_OK


def test_layer_reads_a_weight_written_just_before():
    """Back to back on one stream, each call's operands from the call before."""
    g = gen(9)
    for tokens in (1, 8, 300):
        x = torch.randn(tokens, 2048, generator=g, device="cuda").to(BF16)
        w = torch.randn(2048, 2048, generator=g, device="cuda") * 0.02
        want = ops.fp8_linear(x, ops.fp8_quantize(w, block_rows=128)[0])
        torch.cuda.synchronize()
        for _ in range(20):
            q = ops.fp8_quantize(torch.zeros_like(w), block_rows=128)[0]
            y = ops.fp8_linear(x, ops.fp8_quantize(w, block_rows=128)[0])
            y2 = ops.fp8_linear(x, q)
        assert torch.equal(y, want) and not y2.any()


def test_product_scales_reach_their_ends():
    """Scales 2^-127 .. 2^127 whose products stay in range, and a NaN scale,
    which reaches its row or columns alone."""
    a = ops.fp8_quantize(torch.randn(200, 300, generator=gen(1), device="cuda"))[0]
    b = ops.fp8_quantize(torch.randn(260, 300, generator=gen(2), device="cuda"), block_rows=128)[0]
    a.scale.fill_(0)     # 2^-127
    b.scale.fill_(254)   # 2^127
    near(ops.fp8_matmul(a, b), ref.values(a) @ ref.values(b).t(), product_bound(ref.values(a), ref.values(b), 300))
    few = ops.Fp8Matrix(a.data[:3], a.scale[:, :3].contiguous(), 1)
    near(ops.fp8_matmul(few, b), ref.values(few) @ ref.values(b).t(),
         product_bound(ref.values(few), ref.values(b), 300))
    a.scale.fill_(127)
    b.scale.fill_(127)
    a.scale[1, 7] = 255
    b.scale[2, 1] = 255
    got = ops.fp8_matmul(a, b)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[7] = True
    nan[:, 128:256] = True
    assert torch.equal(torch.isnan(got), nan)
    few = ops.Fp8Matrix(a.data[5:9], a.scale[:, 5:9].contiguous(), 1)
    assert torch.equal(torch.isnan(ops.fp8_matmul(few, b)), nan[5:9])


def test_product_nan_elements_stay_in_their_rows():
    x = torch.randn(140, 200, generator=gen(3), device="cuda")
    x[130, 150] = float("nan")
    w = torch.randn(70, 200, generator=gen(4), device="cuda")
    w[3, 199] = float("inf")
    q, wq = ops.fp8_quantize(x)[0], ops.fp8_quantize(w, block_rows=128)[0]
    got = ops.fp8_matmul(q, wq)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[130] = True
    nan[:, 3] = True
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(torch.isnan(ops.fp8_linear(x[128:132], wq)), nan[128:132])


def test_product_does_not_read_past_its_columns():
    """The bytes between the columns and the next row are never part of the sums."""
    a = ops.fp8_quantize(torch.randn(130, 37, generator=gen(5), device="cuda"))[0]
    full = torch.full((130, 48), 0x7F, dtype=torch.uint8, device="cuda")  # NaN
    full[:, :37] = a.data.view(torch.uint8)
    dirty = ops.Fp8Matrix(full.view(E4)[:, :37], a.scale, 1)
    assert torch.equal(ops.fp8_matmul(dirty, dirty), ops.fp8_matmul(a, a))
    few, clean = (ops.Fp8Matrix(m.data[:2], m.scale[:, :2].contiguous(), 1) for m in (dirty, a))
    assert torch.equal(ops.fp8_matmul(few, dirty), ops.fp8_matmul(clean, a))


def test_product_of_nothing():
    e = ops.fp8_quantize(torch.empty(0, 64, device="cuda"))[0]
    b = ops.fp8_quantize(torch.randn(10, 64, device="cuda"))[0]
    assert ops.fp8_matmul(e, b).shape == (0, 10)
    z = ops.fp8_quantize(torch.empty(10, 0, device="cuda"))[0]
    assert not ops.fp8_matmul(z, z).any()


@pytest.mark.parametrize("tokens,inner,outer,dtype", [(1, 130, 70, BF16), (257, 384, 500, F16), (1030, 256, 129, BF16)])
def test_linear(tokens, inner, outer, dtype):
    g = gen(tokens)
    x = torch.randn(tokens, inner, generator=g, device="cuda").to(dtype)
    w = torch.randn(outer, inner, generator=g, device="cuda") * 0.02
    dy = (torch.randn(tokens, outer, generator=g, device="cuda") * 1e-2).to(dtype)
    q, t = ops.fp8_quantize(w, block_rows=128, transposed=True)
    y = ops.fp8_linear(x.view(1, tokens, inner), q)
    assert y.shape == (1, tokens, outer)
    vx, vw = ref.values(ops.fp8_quantize(x)[0]), ref.values(q)
    want, bound = vx @ vw.t(), product_bound(vx, vw, inner)
    near(y[0], want, bound + (want.abs() + bound) * U[dtype] * 1.01 + TINY[dtype], "y")
    # 8 bits carry 2^-4 of each factor, at random over `inner` terms: an eighth of the result's size
    true = x.double() @ w.double().t()
    assert (y[0].double() - true).norm() <= 0.125 * true.norm()
    dx, dw = ops.fp8_linear_backward(dy, x, t)
    dq, dqt = ops.fp8_quantize(dy, transposed=True)
    vd, vdt, vxt = ref.values(dq), ref.values(dqt), ref.values(ops.fp8_quantize(x, rows=False, transposed=True)[1])
    want, bound = vd @ ref.values(t).t(), product_bound(vd, ref.values(t), outer)
    near(dx, want, bound + (want.abs() + bound) * U[dtype] * 1.01 + TINY[dtype], "dx")
    want, bound = vdt @ vxt.t(), product_bound(vdt, vxt, tokens)
    near(dw, want, bound, "dw")
    twice = dw.clone()
    ops.fp8_linear_backward(dy, x, t, dw=twice, accumulate=True)
    near(twice, 2 * want, 2 * bound + 4 * E * want.abs(), "dw accumulated")


def separate_gradients(dy, x, t, dtype):
    """A layer's gradients as quantisation and two products, one after the other."""
    d, dt = ops.fp8_quantize(dy, transposed=True)
    xt = ops.fp8_quantize(x, rows=False, transposed=True)[1]
    return ops.fp8_matmul(d, t, dtype=dtype), ops.fp8_matmul(dt, xt)


# either product's tiles against the 152 SMs: both fewer, the first fewer, the
# second fewer, both more; cut rows, columns and blocks of K
PAIRS = [(257, 384, 500), (2500, 200, 2500), (2500, 2500, 200), (300, 4100, 3900), (4099, 2048, 6144),
         (5001, 1990, 3001), (3000, 2049, 2047)]


@pytest.mark.parametrize("tokens,inner,outer", PAIRS)
@pytest.mark.parametrize("dtype,fmt", [(BF16, E4), (F16, E5), (F32, E4)])
def test_gradients_are_those_of_the_separate_products(tokens, inner, outer, dtype, fmt):
    """Bit for bit, with gradients of one call after the other in the same
    memory, added to, and read by the call that follows."""
    g = gen(tokens)
    t = ops.fp8_quantize(torch.randn(outer, inner, generator=g, device="cuda") * 0.02, block_rows=128, rows=False,
                         transposed=True, dtype=fmt)[1]
    given = [((torch.randn(tokens, outer, generator=g, device="cuda") * 1e-2).to(dtype),
              torch.randn(tokens, inner, generator=g, device="cuda").to(dtype)) for _ in range(3)]
    want = [separate_gradients(dy, x, t, dtype) for dy, x in given]
    torch.cuda.synchronize()
    sums = [(dx.double().sum(), dw.double().sum()) for dx, dw in want]
    for turn in range(4):
        for (dy, x), (wx, ww), (sx, sw) in zip(given, want, sums):
            dx, dw = ops.fp8_linear_backward(dy, x, t)
            seen = dx.double().sum(), dw.double().sum()
            assert torch.equal(dx, wx) and torch.equal(dw, ww)
            assert torch.equal(seen[0], sx) and torch.equal(seen[1], sw)
            del dx, dw, seen
    total = torch.zeros(outer, inner, device="cuda")
    add = torch.zeros_like(total)
    for (dy, x), (_, ww) in zip(given, want):
        ops.fp8_linear_backward(dy, x, t, dw=total, accumulate=True)
        add += ww
    assert torch.equal(total, add)
    assert ops.status() == B.ROT_OK


def test_gradients_in_a_graph():
    """Both products in one launch, replayed with other inputs, two layers in a row."""
    tokens, inner, outer = 4099, 2048, 2304
    g = gen(12)
    t = ops.fp8_quantize(torch.randn(outer, inner, generator=g, device="cuda") * 0.02, block_rows=128, rows=False,
                         transposed=True)[1]
    back = ops.fp8_quantize(torch.randn(inner, outer, generator=g, device="cuda") * 0.02, block_rows=128, rows=False,
                            transposed=True)[1]
    dy = torch.randn(tokens, outer, generator=g, device="cuda").to(BF16)
    x = torch.randn(tokens, inner, generator=g, device="cuda").to(BF16)

    def step():
        dx, dw = ops.fp8_linear_backward(dy, x, t)
        return (dx, dw, *ops.fp8_linear_backward(dx, dy, back))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(3):
        dy.copy_(torch.randn(tokens, outer, generator=gen(seed), device="cuda"))
        x.copy_(torch.randn(tokens, inner, generator=gen(seed + 10), device="cuda"))
        dx, dw = separate_gradients(dy, x, t, BF16)
        want = (dx, dw, *separate_gradients(dx, dy, back, BF16))
        for _ in range(3):
            for c in captured:
                c.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(want, captured))
    assert ops.status() == B.ROT_OK


def test_layers_of_no_inner_or_outer_features():
    """A last dimension of 0 under any number of leading ones: sums of nothing
    are 0, and the shapes are the leading ones'."""
    def weights(outer, inner):
        return ops.fp8_quantize(torch.zeros(outer, inner, device="cuda"), block_rows=128, transposed=True)

    junk = [torch.full((1 << 16,), float("nan"), device="cuda") for _ in range(8)]
    del junk  # (what an unwritten output would hold)
    for lead in ((3,), (2, 3), (), (2, 1, 5)):
        q, qt = weights(24, 0)
        x = torch.empty(*lead, 0, device="cuda")
        y = ops.fp8_linear(x, q)
        assert y.shape == (*lead, 24) and torch.equal(y, torch.zeros_like(y))
        dy = torch.ones(*lead, 24, device="cuda")
        dx, dw = ops.fp8_linear_backward(dy, x, qt)
        assert dx.shape == x.shape and dw.shape == (24, 0)
        q, qt = weights(0, 24)
        x = torch.ones(*lead, 24, device="cuda")
        assert ops.fp8_linear(x, q).shape == (*lead, 0)
        dx, dw = ops.fp8_linear_backward(torch.empty(*lead, 0, device="cuda"), x, qt)
        assert dx.shape == x.shape and torch.equal(dx, torch.zeros_like(dx)) and dw.shape == (0, 24)
    m, t = ops.fp8_quantize(torch.empty(2, 3, 0, device="cuda"), transposed=True)
    assert m.data.shape == (6, 0) and t.data.shape == (0, 6)
    assert ops.dropout(torch.empty(2, 3, 0, device="cuda"), 0.5, 1).shape == (2, 3, 0)


# ---------------------------------------------------------------------------
# large operands, streams, graphs, all together
# ---------------------------------------------------------------------------


def test_layer_norm_past_2_31_elements():
    """524296 x 4096 in bfloat16: the last rows as by themselves."""
    rows = (1 << 19) + 8
    x = torch.zeros(rows, 4096, dtype=BF16, device="cuda")
    x[-5:] = torch.randn(5, 4096, generator=gen(1), device="cuda").to(BF16)
    w = torch.randn(4096, generator=gen(2), device="cuda")
    y, _, mean, rstd = ops.layer_norm(x, w, w)
    tail = ops.layer_norm(x[-5:], w, w)
    assert torch.equal(y[-5:], tail[0]) and torch.equal(mean[-5:], tail[2])
    dx, _, dw, db = ops.layer_norm_backward(x, x, mean, rstd, w)
    assert torch.equal(dx[-5:], ops.layer_norm_backward(x[-5:], x[-5:], tail[2], tail[3], w)[0])
    del x, y, dx
    torch.cuda.empty_cache()


def test_quantize_and_product_past_2_31_elements():
    """70000 x 32768 to 8 bits in both orientations, and a product of 2.4e9 results."""
    x = torch.zeros(70000, 32768, dtype=BF16, device="cuda")
    x[-300:] = torch.randn(300, 32768, generator=gen(1), device="cuda").to(BF16)
    q, t = ops.fp8_quantize(x, transposed=True)
    first = 70000 // 128 * 128 - 128  # whole blocks of rows
    qa, ta = ops.fp8_quantize(x[first:], transposed=True)
    assert torch.equal(q.data[first:].view(torch.uint8), qa.data.view(torch.uint8))
    assert torch.equal(q.scale[:, first:], qa.scale) and torch.equal(t.scale[first // 128:], ta.scale)
    assert torch.equal(t.data[:, first:].contiguous().view(torch.uint8), ta.data.contiguous().view(torch.uint8))
    del x, q, t
    a = ops.fp8_quantize(torch.randn(40000, 40, generator=gen(2), device="cuda"))[0]
    b = ops.fp8_quantize(torch.randn(60001, 40, generator=gen(3), device="cuda"))[0]
    c = ops.fp8_matmul(a, b, dtype=BF16)
    part = ops.Fp8Matrix(a.data[-130:], a.scale[:, -130:].contiguous(), 1)
    assert torch.equal(c[-130:], ops.fp8_matmul(part, b, dtype=BF16))
    del c
    torch.cuda.empty_cache()


def step_of(x, w, q, qt, targets, ones):
    """A forward and backward pass through one of everything."""
    y, h, mean, rstd = ops.layer_norm(x, w, w, residual=x, p=0.1, seed=3, offset=4)
    logits = ops.fp8_linear(y, q)
    loss, logp, d = ops.policy_loss(logits, targets, -6.0 * ones, ones, ones)
    dy, dw = ops.fp8_linear_backward(d, y, qt)
    return (loss, logp, dw, *ops.layer_norm_backward(dy, h, mean, rstd, w, p=0.1, seed=3, offset=4),
            ops.dropout(x, 0.3, 5, residual=h))


@pytest.mark.parametrize("tokens", [1, 6, 300])
def test_on_another_stream_and_in_a_graph(tokens):
    """The same bits on the current stream, on another one and replayed from a
    graph with new inputs in the captured ones' place."""
    g = gen(tokens)
    x = torch.randn(tokens, 512, generator=g, device="cuda").to(BF16)
    w = torch.ones(512, device="cuda")
    q, qt = ops.fp8_quantize(torch.randn(700, 512, generator=g, device="cuda") * 0.05, block_rows=128, transposed=True)
    targets = torch.randint(700, (tokens,), generator=g, device="cuda")
    args = (x, w, q, qt, targets, torch.ones(tokens, device="cuda"))
    want = step_of(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step_of(*args)
    on = ops.fp8_linear(x, q, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, other)) and torch.equal(on, ops.fp8_linear(x, q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step_of(*args)
    keep = x.clone()
    x.copy_(torch.randn(tokens, 512, generator=g, device="cuda").to(BF16))
    fresh = step_of(*args)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(fresh, captured))
    x.copy_(keep)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, captured))


def test_example_learns():
    """40 steps of the example's bandit, 32 actions: from chance (1 / 32) to
    most rewards."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "policy_step.py")
    spec = importlib.util.spec_from_file_location("policy_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rewards = example.train(steps=40, say=None)
    assert rewards[0] < 0.1 and sum(rewards[-10:]) / 10 > 0.8


# ---------------------------------------------------------------------------
# refusals of the Python entry points
# ---------------------------------------------------------------------------


def test_refusals():
    x = torch.randn(8, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    v = torch.zeros(8, device="cuda")
    t = torch.zeros(8, dtype=torch.int64, device="cuda")
    q, qt = ops.fp8_quantize(x, transposed=True)
    raw = torch.zeros(8 * 64 + 16, dtype=torch.uint8, device="cuda").view(E4)
    for call in (
            lambda: ops.dropout(x.double(), 0.1, 0), lambda: ops.dropout(x.t(), 0.1, 0),
            lambda: ops.dropout(x, 1.5, 0), lambda: ops.dropout(x, 0.1, -1), lambda: ops.dropout(x, 0.1, 1 << 64),
            lambda: ops.dropout(x, 0.1, 0, residual=x[:4]), lambda: ops.dropout(x, 0.1, 0, residual=x.half()),
            lambda: ops.dropout(w.expand(8, 64), 0.1, 0), lambda: ops.dropout(x, 0.1, 0, out=x[:4]),
            lambda: ops.layer_norm(x, w[:32]), lambda: ops.layer_norm(x, w.half()),
            lambda: ops.layer_norm(x, w, w.half()), lambda: ops.layer_norm(x, w, eps=-1.0),
            lambda: ops.layer_norm(x, None), lambda: ops.layer_norm(x, w.cpu()),
            lambda: ops.layer_norm_backward(x, x, v[:4], v, w), lambda: ops.layer_norm_backward(x, x.half(), v, v, w),
            lambda: ops.token_logprobs(x, t.int()), lambda: ops.token_logprobs(x, t[:4]),
            lambda: ops.policy_loss(x, t, v, v, None), lambda: ops.policy_loss(x, t, v, v, v, kl_coef=0.1),
            lambda: ops.policy_loss(x, t, v.double(), v, v), lambda: ops.policy_loss(x, t, v, v, v, out=x.half()),
            lambda: ops.fp8_quantize(x, block_rows=64), lambda: ops.fp8_quantize(x, dtype=torch.uint8),
            lambda: ops.fp8_quantize(x, rows=False), lambda: ops.fp8_matmul(q, qt),
            lambda: ops.fp8_matmul(q, ops.Fp8Matrix(q.data, q.scale[:, :4], 1)),
            lambda: ops.fp8_matmul(q, ops.Fp8Matrix(raw[1:513].view(8, 64), q.scale, 1)),
            lambda: ops.fp8_matmul(q, ops.Fp8Matrix(raw[:8 * 65].view(8, 65)[:, :64], q.scale, 1)),
            lambda: ops.fp8_matmul(q, q, accumulate=True), lambda: ops.fp8_matmul(q, q, dtype=torch.int8),
            lambda: ops.fp8_matmul(q, q, out=torch.empty(8, 9, device="cuda")),
            lambda: ops.fp8_linear(x, w), lambda: ops.fp8_linear_backward(x, x[:4], qt)):
        with pytest.raises((ValueError, B.RotError)):
            call()
