"""Rotary positions and the norm of queries and keys on the GPU against plain
64-bit restatements (tests/heads_adamw_ref.py).

Tolerances.  E = 2^-24, u the unit roundoff of the outputs' type, one rounding
of a result to it costs u |result|.

A cosine or sine: the turn's fraction as float32 is off by E of at most half a
turn (pi E), the function by 2 units in the last place (4 E), the magnitude's
product by E: under 9 E of the magnitude.  Each product and the sum add an E of
their own: a rotated element is off by at most 12 E m (|a| + |b|), a and b its
pair, m the magnitude.

A row's sum of squares adds at most 16 terms one after the other in a lane and
5 over the lanes (22 E), its root halves that; with the products x r w: under
16 E of each element."""

import pytest
import torch

from matrix_optimizer_step_rot_gb300 import binding as B
from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops
from tests import heads_adamw_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 1e-44, F16: 2.0 ** -24, BF16: 1e-39}
E = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    B.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def near(got, want, bound, what=""):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what
    over = ((got - want).abs() - bound)[torch.isfinite(want)]
    assert over.numel() == 0 or over.max().item() <= 0, f"{what}: beyond its bound by {over.max().item():.3e}"


def heads(g, batch, tokens, n, dim, dtype, layout, scale=1.0):
    """[batch, tokens, n, dim] lying in one of several ways, what lies between them NaN."""
    def normal(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    if layout == "fused":  # a part of a wider projection
        x = normal(batch, tokens, n + 3, dim)
        x[:, :, n:] = float("nan")
        return x[:, :, :n]
    if layout == "first":  # heads before tokens
        return normal(batch, n, tokens, dim).transpose(1, 2)
    if layout == "odd":  # heads an odd number of elements apart
        x = normal(batch, tokens, n, dim + 3)
        x[..., dim:] = float("nan")
        return x[..., :dim]
    if layout == "shifted":  # not on a 16-byte boundary
        x = normal(batch * tokens * n * dim + 1)
        return x[1:].view(batch, tokens, n, dim)
    return normal(batch, tokens, n, dim)


def rotary_of(rotated, interleaved, magnitude=1.0, factor=1.0):
    f = ops.rotary_frequencies(rotated, 1e5, factor=factor, original_length=4096)
    return ops.rotary_table(f, magnitude=magnitude, interleaved=interleaved)


# batch, tokens, q heads, k heads (0: none), dim, rotated, interleaved, type, layout, positions
CASES = [
    (1, 1, 1, 0, 2, 2, False, F32, "plain", "start"),
    (1, 1, 16, 8, 128, 128, False, BF16, "plain", "int64"),
    (8, 1, 16, 8, 128, 128, True, BF16, "fused", "int64"),
    (1, 1, 1, 1, 1, 0, False, F32, "plain", "start"),
    (2, 3, 2, 1, 3, 2, False, F16, "plain", "int32"),
    (2, 3, 2, 1, 3, 2, True, BF16, "plain", "int32"),
    (2, 5, 5, 3, 75, 38, True, F32, "plain", "int64"),
    (2, 5, 5, 3, 75, 74, False, F32, "fused", "shared"),
    (1, 7, 4, 4, 72, 72, False, BF16, "plain", "int64"),
    (1, 7, 4, 4, 72, 72, True, BF16, "plain", "int64"),
    (1, 7, 4, 2, 72, 36, False, F16, "plain", "start"),
    (1, 9, 3, 1, 96, 64, True, F16, "fused", "start"),
    (1, 9, 3, 1, 96, 64, False, F16, "first", "shared"),
    (3, 67, 6, 2, 64, 64, False, BF16, "first", "int32"),
    (3, 67, 6, 2, 80, 80, False, BF16, "fused", "int64"),
    (3, 67, 6, 2, 80, 40, True, F32, "first", "int64"),
    (1, 1001, 7, 7, 100, 50, False, BF16, "odd", "int64"),
    (1, 1001, 7, 1, 128, 64, False, BF16, "shifted", "int64"),
    (1, 33, 3, 1, 129, 128, True, F16, "odd", "int64"),
    (1, 33, 3, 2, 200, 200, False, F16, "plain", "int64"),
    (1, 33, 3, 2, 256, 256, False, F32, "plain", "int64"),
    (2, 17, 8, 1, 256, 128, True, F16, "fused", "shared"),
    (1, 33, 3, 2, 264, 264, False, F32, "plain", "int64"),
    (1, 20, 2, 1, 300, 300, False, BF16, "plain", "int64"),
    (1, 20, 2, 1, 301, 150, True, BF16, "plain", "int64"),
    (1, 20, 2, 1, 312, 312, False, F16, "plain", "int64"),
    (1, 20, 2, 1, 512, 512, False, F32, "plain", "int64"),
    (1, 20, 2, 1, 512, 512, True, F32, "fused", "int64"),
    (1, 20, 2, 2, 512, 256, False, BF16, "plain", "int64"),
    (1, 20, 2, 2, 511, 510, False, F32, "plain", "int64"),
    (1, 20, 2, 2, 509, 508, True, F16, "plain", "int64"),
    (1, 4, 65, 33, 16, 16, False, BF16, "plain", "int64"),
    (1, 4, 65, 33, 8, 8, True, BF16, "plain", "int64"),
    (1, 300, 1, 0, 128, 0, False, BF16, "plain", "start"),
    (2, 31, 5, 2, 100, 100, False, BF16, "plain", "int64"),
    (1, 31, 5, 2, 196, 196, False, F16, "fused", "int64"),
    (1, 31, 3, 1, 500, 500, False, BF16, "plain", "int64"),
    (2, 40, 3, 2, 22, 20, False, F16, "first", "int64"),
    (1, 40, 9, 5, 128, 128, False, BF16, "plain", "int64"),  # groups past the last head
    (1, 2900, 9, 5, 128, 128, True, F16, "fused", "int64"),
    (1, 700, 1, 1, 256, 128, False, BF16, "first", "int32"),
    (1, 1, 300, 7, 512, 512, False, F32, "plain", "int64"),  # one token's heads over many warps
    (1, 2, 1000, 1, 40, 20, True, BF16, "odd", "int64"),
    (1, 1, 4000, 500, 128, 128, False, BF16, "plain", "start"),
    (3, 700, 1, 1, 128, 128, False, BF16, "plain", "int64"),  # a few more tokens than warps
    (2, 2500, 16, 8, 128, 128, False, BF16, "fused", "int64"),
    (1, 3000, 3, 3, 40, 20, True, F16, "fused", "int32"),
]


def inputs(case, seed):
    batch, tokens, q, k, dim, rotated, interleaved, dtype, layout, where = case
    g = gen(seed)
    x = heads(g, batch, tokens, q, dim, dtype, layout)
    y = heads(g, batch, tokens, k, dim, dtype, layout) if k else None
    rotary = rotary_of(rotated, interleaved, 1.0 if q % 2 else 1.25, 4.0 if dim % 3 else 1.0)
    at = torch.arange(tokens, device="cuda").expand(batch, tokens)
    kw = {}
    if where == "start":
        kw["start"], at = 70001, at + 70001
    elif where == "shared":
        at = torch.randint(1 << 20, (tokens,), generator=g, device="cuda")
        kw["positions"], at = at, at.expand(batch, tokens)
    else:
        at = torch.randint(-5, 1 << 30, (batch, tokens), generator=g, device="cuda")
        kw["positions"] = at.to(torch.int32 if where == "int32" else torch.int64)
    return g, x, y, rotary, at, kw


def rotation_bound(x, want, rotary, dtype):
    return 12 * E * ref.pair_size(x, rotary) + U[dtype] * want.abs() * 1.01 + TINY[dtype]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_rotate(case, inverse):
    g, x, y, rotary, at, kw = inputs(case, 1)
    call = ops.rotate_backward if inverse else ops.rotate
    got, got_k = call(x, rotary, y, **kw)
    for a, b in ((x, got), (y, got_k)):
        if a is None:
            assert b is None
            continue
        want = ref.rotated(a, rotary, at, inverse)
        near(b, want, rotation_bound(a, want, rotary, a.dtype))
        assert torch.equal(b[..., case[5]:], a[..., case[5]:])  # what is not rotated
    # into views of the inputs' own layout, and in place
    o = heads(g, *x.shape[:3], x.shape[3], x.dtype, case[8])
    rest = o.untyped_storage().nbytes()
    assert call(x, rotary, out=o, **kw)[0] is o and torch.equal(o, got) and o.untyped_storage().nbytes() == rest
    keep = x.clone()
    z = x.as_strided(x.shape, x.stride(), x.storage_offset())
    call(z, rotary, out=z, **kw)
    assert torch.equal(z, got) and not (case[5] and torch.equal(keep, got) and at.abs().max() > 0)


@pytest.mark.parametrize("case", CASES)
def test_head_norm(case):
    g, x, y, rotary, at, kw = inputs(case, 2)
    dim, dtype = case[4], case[7]
    wtype = dtype if case[2] % 3 == 0 else F32
    w = [(1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(wtype) for _ in range(2)]
    for r in (rotary, None):
        more = dict(kw, rotary=r) if r is not None else {}
        got, got_k = ops.head_norm(x, w[0], y, w[1] if y is not None else None, EPS, **more)
        for a, b, v in ((x, got, w[0]), (y, got_k, w[1])):
            if a is None:
                assert b is None
                continue
            flat = ref.normed(a, v, EPS)[0]
            want = flat if r is None else ref.rotated(flat, r, at)
            near(b, want, (12 + 16) * E * ref.pair_size(flat, r) + U[dtype] * want.abs() * 1.01 + TINY[dtype])
    z = x.as_strided(x.shape, x.stride(), x.storage_offset())
    ops.head_norm(z, w[0], eps=EPS, out=z)
    assert torch.equal(z, got)


@pytest.mark.parametrize("case", CASES)
def test_head_norm_backward(case):
    """dx = r (g w - hat mean(g w hat)): g is off by 12 E G, G the pair's size
    in dy, hat by 16 E, the mean's sum by 22 E and its terms' own errors (12 +
    16 + 2); the rest is products."""
    g, x, y, rotary, at, kw = inputs(case, 3)
    batch, tokens, q, k, dim, _, _, dtype, _, _ = case
    wtype = dtype if case[2] % 3 == 0 else F32
    w = [(1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(wtype) for _ in range(2)]
    d = [heads(g, batch, tokens, q, dim, dtype, "plain", 1e-2),
         heads(g, batch, tokens, k, dim, dtype, "first", 1e-2) if k else None]
    for r in (rotary, None):
        more = dict(kw, rotary=r) if r is not None else {}
        dq, dk, dwq, dwk = ops.head_norm_backward(d[0], x, w[0], d[1], y, w[1] if k else None, EPS, **more)
        for dy, a, v, dx, dw, n in ((d[0], x, w[0], dq, dwq, q), (d[1], y, w[1], dk, dwk, k)):
            if a is None:
                assert dx is None and dw is None
                continue
            back = dy.double() if r is None else ref.rotated(dy, r, at, True)
            want, want_w = ref.norm_grad(back, a, v, EPS)
            _, hat, rstd = ref.normed(a, v, EPS)
            size = ref.pair_size(dy, r) * v.double().abs()
            bound = rstd * (30 * E * size + 80 * E * hat.abs() * (size * hat.abs()).mean(-1, keepdim=True))
            near(dx, want, bound + 20 * E * want.abs() + U[dtype] * want.abs() * 1.01 + TINY[dtype])
            # the weight's sum: a lane's heads and tokens one after the other, then at most 5 + 3 + 32 + 5
            chain = 48 + n + batch * tokens * n // 1500
            total = (ref.pair_size(dy, r) * hat.abs()).flatten(0, -2).sum(0)
            near(dw, want_w, (12 + 16 + chain) * E * total + 1e-30)
    # in place (queries alone: other blocks, so that the weight's sum has another order)
    z = d[0].clone()
    got, alone = ops.head_norm_backward(z, x, w[0], eps=EPS, out=z), ops.head_norm_backward(d[0], x, w[0], eps=EPS)
    assert got[0] is z and torch.equal(z, dq) and torch.equal(got[2], alone[2])
    assert got[1] is None and got[3] is None


def test_gradients_against_differences():
    """Float64 central differences of the 64-bit forward pass, which the kernel's forward pass is held to above."""
    g = gen(4)
    x = torch.randn(2, 3, 2, 12, generator=g, device="cuda")
    w = 1 + 0.2 * torch.randn(12, generator=g, device="cuda")
    dy = torch.randn(2, 3, 2, 12, generator=g, device="cuda")
    rotary, at = rotary_of(8, True, 1.5), torch.arange(3, device="cuda").expand(2, 3) + 11

    def loss(x, w):
        return (ref.rotated(ref.normed(x, w, EPS)[0], rotary, at) * dy.double()).sum().item()

    dx, _, dw, _ = ops.head_norm_backward(dy, x, w, eps=EPS, rotary=rotary, start=11)
    h = 1e-5
    for i in range(0, x.numel(), 5):
        e = torch.zeros(x.numel(), dtype=torch.float64, device="cuda")
        e[i] = h
        e = e.view(x.shape)
        want = (loss(x.double() + e, w.double()) - loss(x.double() - e, w.double())) / (2 * h)
        assert abs(dx.flatten()[i].item() - want) <= 1e-5 * (1 + abs(want))  # (h^2 and 2^-24 of sums of a few units)
    for i in range(12):
        e = torch.zeros(12, dtype=torch.float64, device="cuda")
        e[i] = h
        want = (loss(x.double(), w.double() + e) - loss(x.double(), w.double() - e)) / (2 * h)
        assert abs(dw[i].item() - want) <= 1e-5 * (1 + abs(want))


@pytest.mark.parametrize("position", [0, 1, 12345, 10 ** 6 + 7, 2 ** 31 - 1, 2 ** 31 + 12345, -77, 10 ** 12])
def test_angles_of_far_positions(position):
    """cos and sin of position times frequency, by whole numbers of 2^-64 of a
    turn worked out in Python (the frequency itself is a float64, and its turn's
    rounding to 2^-64 costs position 2^-64 of a turn)."""
    import math
    from fractions import Fraction

    pi = Fraction(3141592653589793238462643383279502884197, 10 ** 39)
    f = ops.rotary_frequencies(64, 10000.0)
    rotary = ops.rotary_table(f)
    x = torch.zeros(1, 1, 64, device="cuda")
    x[..., :32] = 1.0
    got = ops.rotate(x, rotary, positions=torch.tensor([position], device="cuda"))[0].double().flatten().tolist()
    for i, v in enumerate(f.tolist()):
        turn = Fraction(v) * position / (2 * pi)
        a = 2 * math.pi * float(turn - math.floor(turn))
        # float64's 2^-53 of the frequency over 2 pi, times the position
        bound = 12 * E * 2 + abs(position) * 2.0 ** -52 * v
        assert abs(got[i] - math.cos(a)) <= bound and abs(got[32 + i] - math.sin(a)) <= bound


def test_rows_between_the_heads_are_left_alone():
    g = gen(6)
    buffer = torch.randn(50, 10, 64, generator=g, device="cuda").bfloat16()
    keep = buffer.clone()
    rotary, w = rotary_of(64, False), torch.ones(64, device="cuda")
    q, k = buffer[:40, :4], buffer[:40, 4:6]  # tokens 40 to 49 are padding, heads 6 to 9 the values
    ops.head_norm(q, w, k, w, rotary=rotary, out=q, k_out=k)
    assert torch.equal(buffer[40:], keep[40:]) and torch.equal(buffer[:, 6:], keep[:, 6:])
    want = ops.head_norm(keep[:40, :4], w, keep[:40, 4:6], w, rotary=rotary)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_three_dimensions_and_shared_inputs():
    """[tokens, heads, dim] is one batch entry; inputs may be expanded; results do not depend on the launch's split."""
    g = gen(7)
    x = torch.randn(9, 4, 64, generator=g, device="cuda")
    rotary, at = rotary_of(64, True), torch.randint(9999, (9,), generator=g, device="cuda")
    w = torch.rand(64, generator=g, device="cuda")
    a = ops.head_norm(x, w, rotary=rotary, positions=at)[0]
    assert torch.equal(a, ops.head_norm(x[None], w, rotary=rotary, positions=at)[0][0])
    assert torch.equal(a, ops.head_norm(x[None], w, rotary=rotary, positions=at[None])[0][0])
    b = ops.head_norm(x.expand(500, 9, 4, 64), w, rotary=rotary, positions=at)[0]
    assert torch.equal(b, a.expand(500, 9, 4, 64))
    c = ops.rotate(x[:1].expand(9, 4, 64), rotary, positions=at[:1].expand(9))[0]
    assert torch.equal(c, ops.rotate(x[:1], rotary, positions=at[:1])[0].expand(9, 4, 64))
    d = ops.head_norm_backward(a, x, w, rotary=rotary, positions=at)
    assert all(torch.equal(u, v) for u, v in zip(d[::2], ops.head_norm_backward(a, x, w, rotary=rotary,
                                                                                positions=at)[::2]))


def test_nothing_there():
    rotary, w = rotary_of(64, False), torch.ones(64, device="cuda")
    for shape in ((0, 4, 64), (5, 0, 64), (0, 5, 4, 64), (2, 0, 4, 64)):
        x = torch.empty(shape, device="cuda")
        assert ops.rotate(x, rotary)[0].shape == x.shape
        assert ops.head_norm(x, w, x, w, rotary=rotary)[1].shape == x.shape
        dq, dk, dw, dv = ops.head_norm_backward(x, x, w, x, x, w, rotary=rotary)
        assert dq.shape == x.shape and torch.equal(dw, torch.zeros(64, device="cuda")) and torch.equal(dw, dv)
    # keys alone are there
    x, y = torch.empty(5, 0, 64, device="cuda"), torch.randn(5, 2, 64, device="cuda")
    q, k = ops.rotate(x, rotary, y, start=3)
    assert q.shape == x.shape and torch.equal(k, ops.rotate(y, rotary, start=3)[0])
    dq, dk, dw, dv = ops.head_norm_backward(x, x, w, y, y, w)
    one = ops.head_norm_backward(y, y, w)
    assert torch.equal(dk, one[0]) and torch.equal(dv, one[2]) and dw.abs().max() == 0


@pytest.mark.parametrize("dim,rotated,interleaved", [(128, 64, False), (128, 64, True), (75, 38, False)])
def test_special_values_stay_in_their_heads(dim, rotated, interleaved):
    """A NaN or an infinity reaches its own pair (rotate) or head (norm) alone; a head of zeros gives zeros."""
    g = gen(8)
    x = torch.randn(3, 4, dim, generator=g, device="cuda")
    x[0, 1, 3], x[1, 2, dim - 1], x[2, 3] = float("nan"), float("inf"), 0.0
    rotary, w = rotary_of(rotated, interleaved), torch.ones(dim, device="cuda")
    got = ops.rotate(x, rotary, start=5)[0]
    want = ref.rotated(x, rotary, torch.arange(3, device="cuda") + 5)
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)) and got[1, 2, dim - 1].item() == float("inf")
    y = ops.head_norm(x, w, rotary=rotary, start=5)[0]
    assert torch.isnan(y[0, 1]).all() and torch.isnan(y[1, 2]).any() and y[2, 3].abs().max() == 0
    for t, h in ((0, 1), (1, 2)):
        y[t, h] = 0
    assert torch.isfinite(y).all()
    dx, _, dw, _ = ops.head_norm_backward(torch.ones_like(x), x, w, rotary=rotary, start=5)
    assert torch.isfinite(dx[2, 3]).all() and torch.isfinite(dx[0, 0]).all() and torch.isnan(dw).any()
    # no eps: only heads of zeros are undefined
    y = ops.head_norm(x, w, eps=0.0)[0]
    assert torch.isnan(y[2, 3]).all() and torch.isfinite(y[2, 2]).all()
    one = x[2, :3].clone()[None]  # (three heads to groups of lanes: the idle ones give the sums nothing)
    assert torch.isfinite(ops.head_norm_backward(torch.ones_like(one), one, w, eps=0.0)[2]).all()


def test_past_2_31_elements():
    """Offsets beyond 32 bits, in the input and the output."""
    tokens, n, dim = 70000, 64, 512
    x = torch.zeros(tokens, n, dim, dtype=BF16, device="cuda")
    part = torch.randn(3, n, dim, generator=gen(9), device="cuda").to(BF16)
    for at in (0, 65536, tokens - 3):
        x[at:at + 3] = part
    rotary, w = rotary_of(512, False), torch.ones(dim, device="cuda")
    at = torch.arange(tokens, device="cuda")
    at[65536:65539] = at[tokens - 3:] = torch.arange(3, device="cuda")
    y = ops.head_norm(x, w, rotary=rotary, positions=at)[0]
    want = ops.head_norm(part, w, rotary=rotary)[0]
    for i in (0, 65536, tokens - 3):
        assert torch.equal(y[i:i + 3], want)
    ops.rotate(x, rotary, positions=at, out=x)
    assert torch.equal(x[tokens - 3:], ops.rotate(part, rotary)[0])
    ops.head_norm_backward(y, x, w, rotary=rotary, positions=at, out=y)
    assert torch.equal(y[tokens - 3:], ops.head_norm_backward(want, x[:3], w, rotary=rotary)[0])
    del x, y
    torch.cuda.empty_cache()


def test_streams_and_graphs():
    """The same bits on another stream, and replayed with new inputs in the captured ones' place."""
    g = gen(10)
    x = torch.randn(1, 40, 24, 128, generator=g, device="cuda").bfloat16()
    d = torch.randn(1, 40, 24, 128, generator=g, device="cuda").bfloat16()
    at = torch.arange(40, device="cuda")[None] + 500
    w, v = torch.rand(128, generator=g, device="cuda"), torch.rand(128, generator=g, device="cuda")
    rotary = rotary_of(128, False)

    def run(stream=None):
        q, k = x[:, :, :16], x[:, :, 16:]
        a = ops.rotate(q, rotary, k, positions=at, stream=stream)
        b = ops.head_norm(q, w, k, v, rotary=rotary, positions=at, stream=stream)
        c = ops.head_norm_backward(d[:, :, :16], q, w, d[:, :, 16:], k, v, rotary=rotary, positions=at, stream=stream)
        e = ops.rotate_backward(d[:, :, :16], rotary, d[:, :, 16:], positions=at, stream=stream)
        return [*a, *b, *c, *e]

    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = run(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    with torch.cuda.graph(second, pool=graph.pool()):
        again = run()
    x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    at += 1000
    fresh = run()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(fresh, captured))
    second.replay()
    assert all(torch.equal(a, b) for a, b in zip(fresh, again))


def test_two_threads_at_once():
    """Calls of two threads, each on a stream of its own: the same bits as alone."""
    import threading

    w, rotary = torch.rand(128, generator=gen(12), device="cuda"), rotary_of(128, True)
    xs = [torch.randn(200, 6, 128, generator=gen(30 + i), device="cuda").bfloat16() for i in range(2)]

    def work(x, stream=None):
        y = ops.head_norm(x, w, x, w, rotary=rotary, start=9, stream=stream)
        return [*y, *ops.head_norm_backward(y[0], x, w, y[1], x, w, rotary=rotary, start=9, stream=stream)]

    want, got = [work(x) for x in xs], [None, None]
    torch.cuda.synchronize()

    def run(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i] = work(xs[i], s)
        s.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(a, b) for p, q in zip(want, got) for a, b in zip(p, q))


def test_refusals():
    x = torch.randn(2, 5, 4, 64, device="cuda")
    w, rotary = torch.ones(64, device="cuda"), rotary_of(64, False)
    p = torch.zeros(2, 5, dtype=torch.int64, device="cuda")
    turns = rotary.turns
    for call in (
            lambda: ops.rotate(x.cpu(), rotary), lambda: ops.rotate(x.double(), rotary), lambda: ops.rotate(x[0, 0], rotary),
            lambda: ops.rotate(x.transpose(2, 3), rotary), lambda: ops.rotate(x, None), lambda: ops.rotate(x, turns),
            lambda: ops.rotate(x, rotary_of(66, False)), lambda: ops.rotate(x, ops.Rotary(turns.int())),
            lambda: ops.rotate(x, ops.Rotary(turns.cpu())), lambda: ops.rotate(x, ops.Rotary(turns, float("nan"))),
            lambda: ops.rotate(x, ops.Rotary(turns[::2])), lambda: ops.rotate(x, rotary, x.half()),
            lambda: ops.rotate(x, rotary, x[:, :3]), lambda: ops.rotate(x, rotary, x[..., :32]),
            lambda: ops.rotate(x, rotary, positions=p.float()), lambda: ops.rotate(x, rotary, positions=p[:, :4]),
            lambda: ops.rotate(x, rotary, positions=p[:1]), lambda: ops.rotate(x, rotary, positions=p.cpu()),
            lambda: ops.rotate(x, rotary, out=x[:, :, :3]), lambda: ops.rotate(x, rotary, out=x.half()),
            lambda: ops.rotate(x, rotary, k_out=x), lambda: ops.rotate(x, rotary, out=x[:, :1].expand(2, 5, 4, 64)),
            lambda: ops.rotate(torch.zeros(2, 2, 600, device="cuda"), rotary),
            lambda: ops.head_norm(x, w[:32]), lambda: ops.head_norm(x, w.double()), lambda: ops.head_norm(x, None),
            lambda: ops.head_norm(x, w, x), lambda: ops.head_norm(x, w, None, w), lambda: ops.head_norm(x, w, eps=-1.0),
            lambda: ops.head_norm(x.half(), w, x.half(), w.half()), lambda: ops.head_norm(x, w, rotary=turns),
            lambda: ops.head_norm(x, w, eps=float("nan")), lambda: ops.head_norm_backward(x, x[:, :, :3], w),
            lambda: ops.head_norm_backward(x, x.half(), w), lambda: ops.head_norm_backward(x, x, w, x, x),
            lambda: ops.head_norm_backward(x, x, w, None, x, w), lambda: ops.head_norm_backward(x, x, w, k_out=x)):
        with pytest.raises((ValueError, B.RotError)):
            call()
