"""AdamW over many tensors and the gradient's norm on the GPU against plain
64-bit restatements (tests/heads_adamw_ref.py).

Tolerances, E = 2^-24.  m: two products of rounded factors and their sum, 4 E
(|beta1 m| + |(1 - beta1) g|).  v: all terms are positive, 6 E v; its root 4 E.
p: the decay's factor and product 2 E |p|, the update (root, correction, eps,
quotient: the fast division is good to 2 units in the last place) 16 E |u| on
top of m's error, the difference E.  Where a number lands on a grid at random,
its place between two neighbours may differ by the float32 error: only then the
other neighbour counts."""

import numpy as np
import pytest
import torch

from matrix_optimizer_step_rot_gb300 import binding as B
from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops
from matrix_optimizer_step_rot_gb300.optimizer import AdamW, RotatedAdam
from tests import heads_adamw_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E4 = torch.float8_e4m3fn
E = 2.0 ** -24
SEED = 0xFEDCBA9876543210
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-7, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    B.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def shifted(t, by):
    """t's values `by` elements behind an aligned address."""
    flat = torch.zeros(t.numel() + by, dtype=t.dtype, device=t.device)
    if t.dtype == E4:
        flat.view(torch.uint8)[by:] = t.view(torch.uint8).flatten()
    else:
        flat[by:] = t.flatten()
    return flat[by:].view(t.shape)


def lists(sizes, ptype, gtype, master, bits, seed, shift=0):
    """Parameters, gradients and states as after some steps."""
    g = gen(seed)
    out = dict(p=[], g=[], m=[], v=[], master=[])
    for n in sizes:
        w = torch.randn(n, generator=g, device="cuda") * 0.05
        out["p"].append(shifted(w.to(ptype), shift))
        out["master"].append(shifted(w, shift) if master else None)
        spread = torch.exp(2.0 * torch.randn(n, generator=g, device="cuda"))
        out["g"].append(shifted((torch.randn(n, generator=g, device="cuda") * 1e-3 * spread).to(gtype), shift))
        m, v = torch.randn(n, generator=g, device="cuda") * 1e-3, torch.rand(n, generator=g, device="cuda") * 1e-5
        if bits == 32:
            out["m"].append(shifted(m, shift))
            out["v"].append(shifted(v, shift))
        else:
            for name, x in (("m", m), ("v", v.sqrt())):
                x = x.cpu().double().numpy()
                e = ref.scale_exponents(x)
                q = torch.from_numpy(x * 2.0 ** -e).float().to(E4)
                scale = torch.from_numpy((e[::128] + 127).astype(np.uint8))
                out[name].append(ops.Fp8Vector(shifted(q.cuda(), shift), scale.cuda()))
    return out


def f64(t):
    return (t.dequantize() if isinstance(t, ops.Fp8Vector) else t).double().cpu().numpy().reshape(-1)


def on_grid(got, value, error, step, part, what):
    """got is floor(|value| / step + part) steps, or what it is anywhere within value's error: the other neighbour
    where that reaches the border, and any step between the ends where a difference that cancels leaves a number
    whose own steps are smaller than its error (p = 1e-7 of two numbers of 0.05: error 3e-9, steps of 5e-10)."""
    place = np.abs(value) / step + part
    wide = error / step + 1e-12
    low, high = np.floor(place - wide), np.floor(place + wide)
    have = np.abs(got) / step
    beside = (have < low) | (have > high)
    assert not beside.any(), f"{what}: beside the grid: {[a[beside][:3] for a in (got, value, error, step, part)]}"
    assert np.sum(low != high) <= 2 + 0.01 * len(value), what  # (of which there are few)
    assert np.all((np.sign(got) == np.sign(value)) | (got == 0) | (np.abs(value) < error)), what


def check(before, after, t, factor=1.0, hyper=HYPER, rounded=True):
    base = 0
    for i in range(len(before["p"])):
        n = before["p"][i].numel()
        w = ref.words(base, n, t, SEED)
        base += -(-n // 128) * 128
        if n == 0:
            continue
        eight = isinstance(before["m"][i], ops.Fp8Vector)
        g, m, v = f64(before["g"][i]), f64(before["m"][i]), f64(before["v"][i])
        v = v * v if eight else v
        start = before["master"][i] if before["master"][i] is not None else before["p"][i]
        p, nm, nv = ref.step(f64(start), g, m, v, t, hyper["lr"], hyper["beta1"], hyper["beta2"], hyper["eps"],
                             hyper["weight_decay"], factor)
        fg = np.abs(g * factor)
        merr = 4 * E * (np.abs(hyper["beta1"] * m) + (1 - hyper["beta1"]) * fg) * (1 if factor == 1.0 else 1.5) + 1e-45
        u = np.abs(f64(start) * (1 - hyper["lr"] * hyper["weight_decay"]) - p)
        with np.errstate(divide="ignore", invalid="ignore"):
            perr = np.where(nm != 0, u / np.abs(nm), 0.0) * merr + 16 * E * u + 3 * E * np.abs(f64(start)) + 1e-45
        if eight:
            part = ((w & 0xFFFF) + 0.5) / 65536
            for name, x, err in (("m", nm, merr), ("v", np.sqrt(nv), 5 * E * np.sqrt(nv))):
                got = after[name][i]
                e = ref.scale_exponents(x)
                top = np.maximum.reduceat(np.abs(x), np.arange(0, n, 128))
                border = np.abs(np.log2(top / 448.0) - np.round(np.log2(np.maximum(top, 1e-300) / 448.0))) < 1e-6
                have = got.scale.cpu().numpy().astype(np.float64) - 127
                assert np.all((have == e[::128]) | border), name
                e = np.repeat(have, 128)[:n]
                step = ref.grid(x, e, 3, -6)
                val = f64(got)
                if name == "v":  # a root above 0 is not 0
                    least = 2.0 ** (e - 9)
                    assert np.all(val[x > 1e-40] >= least[x > 1e-40])
                    small = np.abs(x) / step + part < 1
                    val = np.where(small & (val == least), 0.0, val)
                on_grid(val, x, err, step, part, name)
        else:
            assert np.all(np.abs(f64(after["m"][i]) - nm) <= merr), "m"
            assert np.all(np.abs(f64(after["v"][i]) - nv) <= 6 * E * nv * (1 if factor == 1.0 else 1.5) + 1e-45), "v"
        if before["master"][i] is not None:
            assert np.all(np.abs(f64(after["master"][i]) - p) <= perr), "master"
            assert torch.equal(after["p"][i], after["master"][i].to(after["p"][i].dtype)), "copy"
        elif before["p"][i].dtype == BF16:
            part = (w >> 16) / 65536
            on_grid(f64(after["p"][i]), p, perr, ref.grid(p, np.zeros(n), 7, -126), part, "p")
        else:
            assert np.all(np.abs(f64(after["p"][i]) - p) <= perr), "p"


def cloned(x):
    return {k: [ops.Fp8Vector(t.data.clone(), t.scale.clone()) if isinstance(t, ops.Fp8Vector)
                else None if t is None else t.clone() for t in v] for k, v in x.items()}


def call(x, t, **kw):
    ops.adamw(x["p"], x["g"], x["m"], x["v"], t, masters=x["master"], seed=SEED, **dict(HYPER, **kw))


def same(a, b):
    for k in a:
        for s, t in zip(a[k], b[k]):
            if isinstance(s, ops.Fp8Vector):
                if not (torch.equal(s.data.view(torch.uint8), t.data.view(torch.uint8)) and torch.equal(s.scale, t.scale)):
                    return False
            elif s is not None and not torch.equal(s, t):
                return False
    return True


KINDS = [(F32, F32, False), (F32, BF16, False), (BF16, BF16, False), (BF16, F32, False), (BF16, F16, False),
         (BF16, BF16, True), (BF16, F32, True), (F16, F16, True), (F16, F32, True)]
SIZES = [[1], [4096], [3, 0, 127, 128, 129, 5000, 1], [12289, 4095, 4097, 70001], [64] * 40, [300] * 800]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("ptype,gtype,master", KINDS)
def test_step(ptype, gtype, master, bits, shift):
    for k, sizes in enumerate(SIZES if not shift else SIZES[2:4]):
        x = lists(sizes, ptype, gtype, master, bits, 10 * k + bits, shift)
        before = cloned(x)
        call(x, 7 + k)
        check(before, x, 7 + k)
        call(before, 7 + k)
        assert same(before, x)  # again, bit for bit


def test_mixed_lists():
    """Types, masters and states of all kinds in one call: each as in a call of its own at its place in the list."""
    parts = [lists([n], *kind, bits, n) for n, (kind, bits) in enumerate([(k, b) for k in KINDS for b in (32, 8)], 100)]
    x = {k: [t for part in parts for t in part[k]] for k in parts[0]}
    before = cloned(x)
    call(x, 3)
    check(before, x, 3)


def test_first_steps_from_nothing():
    """Zeros as states, four steps."""
    for bits in (32, 8):
        x = lists([1000, 130], F32, F32, False, 32, 5)
        for k in ("m", "v"):
            x[k] = [ops.adamw_state(p, bits=bits)[k == "v"] for p in x["p"]]
        for t in range(1, 5):
            before = cloned(x)
            call(x, t)
            check(before, x, t)


@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_and_scale(bits):
    x = lists([5000, 77], F32, F32, False, bits, 6)
    flat = np.concatenate([f64(g) for g in x["g"]])
    norm = ops.gradient_norm(x["g"])
    assert abs(norm.item() - np.linalg.norm(flat)) <= 64 * E * norm.item()
    for scale, max_norm in ((1.0, 1e-3), (1.0, 1e9), (0.25, 1e-3), (-3.0, 1e-2), (0.5, 1e9)):
        y = cloned(x)
        before = cloned(x)
        call(y, 9, norm=norm, max_norm=max_norm, scale=scale)
        factor = scale * min(1.0, max_norm / (abs(scale) * norm.item()))
        check(before, y, 9, factor)
    # no step where the norm is not finite
    for bad in (float("nan"), float("inf")):
        y = cloned(x)
        call(y, 9, norm=torch.tensor(bad, device="cuda"))
        assert same(x, y)


def test_step_and_rate_on_the_device():
    """The corrections 1 - beta^t by expm1 there, by pow on the host: 1 - beta^t is off by 4 E t |log beta| at most
    of the exponent and E of itself, relative to it (t |log beta| / (1 - beta^t) < 1 + t |log beta|)."""
    for t in (1, 2, 10, 1000, 100000):
        x = lists([5000], F32, F32, False, 32, 8)
        y, z = cloned(x), cloned(x)
        call(x, t)
        call(y, torch.tensor([t], device="cuda"), lr=torch.tensor(1e-2, device="cuda"))
        u = (z["p"][0].double() * (1 - 1e-3) - x["p"][0].double()).abs()
        assert ((x["p"][0].double() - y["p"][0].double()).abs()
                <= 64 * E * u + 4 * E * x["p"][0].double().abs() + 2 * E * z["p"][0].double().abs()).all()
        assert torch.equal(x["m"][0], y["m"][0])
    call(z, torch.zeros(1, dtype=torch.int64, device="cuda"))  # no step 0
    assert same(z, lists([5000], F32, F32, False, 32, 8))
    # the same random words
    x = lists([5000], BF16, BF16, False, 8, 8)
    y = cloned(x)
    call(x, 6)
    call(y, torch.tensor(6, device="cuda"))
    assert all(torch.equal(x[k][0].scale, y[k][0].scale) for k in "mv")
    assert (x["p"][0] != y["p"][0]).double().mean() < 0.01


def test_special_values():
    """NaN and infinities stay in their places; the rest of their 128 goes on as without them."""
    for bits in (32, 8):
        x = lists([512], F32, F32, False, bits, 11)
        clean = cloned(x)
        for at, bad in ((5, float("nan")), (130, float("inf")), (131, float("-inf"))):
            x["g"][0][at] = bad
            clean["g"][0][at] = 0.0
        call(x, 4)
        call(clean, 4)
        odd = torch.zeros(512, dtype=torch.bool, device="cuda")
        odd[[5, 130, 131]] = True
        assert torch.equal(torch.isnan(x["p"][0]), odd)
        assert torch.equal(x["p"][0][~odd], clean["p"][0][~odd])
        if bits == 8:
            assert torch.equal(torch.isnan(x["m"][0].dequantize()), odd)
            assert torch.equal(torch.isnan(x["v"][0].dequantize()), odd)
        # bfloat16 parameters without a master, aligned and not
        for shift in (0, 1):
            y = lists([512], BF16, F32, False, bits, 11, shift)
            for at, bad in ((5, float("nan")), (130, float("inf")), (131, float("-inf"))):
                y["g"][0][at] = bad
            y["p"][0][200], y["p"][0][201] = float("inf"), float("-inf")
            keep = y["p"][0].clone()
            call(y, 4)
            odd[[5, 130, 131]] = True
            assert torch.equal(torch.isnan(y["p"][0]), odd)
            assert y["p"][0][200].item() == float("inf") and y["p"][0][201].item() == float("-inf")
            assert torch.isfinite(y["p"][0][~odd]).sum() == 512 - 5 and (y["p"][0] != keep).sum() > 300
        # a tensor of zero gradients and states moves by its decay alone
        z = lists([300], F32, F32, False, 32, 12)
        z["g"][0].zero_()
        z["m"], z["v"] = ([ops.adamw_state(z["p"][0], bits=bits)[k]] for k in (0, 1))
        keep = z["p"][0].clone()
        call(z, 1)
        near = (z["p"][0].double() - keep.double() * (1 - 1e-3)).abs()
        assert (near <= 2 * E * keep.double().abs()).all() and f64(z["v"][0]).max() == 0


def test_extreme_scales_in_8_bits():
    """Moments from 2^-140 to 2^100 in their blocks: scale bytes at both ends of their range."""
    n = 128 * 40
    g = torch.randn(n, generator=gen(13), device="cuda").view(40, 128)
    g = (g * torch.exp2(torch.linspace(-60, 60, 40, device="cuda"))[:, None]).flatten()
    x = dict(p=[torch.zeros(n, device="cuda")], g=[g], m=[], v=[], master=[None])
    for k in (0, 1):
        x["mv"[k]].append(ops.adamw_state(x["p"][0], bits=8)[k])
    before = cloned(x)
    call(x, 1, beta1=0.0, beta2=0.0)
    hyper = dict(HYPER, beta1=0.0, beta2=0.0)
    check(before, x, 1, hyper=hyper)
    tiny = torch.full((256,), 1e-42, device="cuda")
    tiny[:128] = 3e38
    x = dict(p=[torch.zeros(256, device="cuda")], g=[tiny], m=[ops.adamw_state(tiny, bits=8)[0]],
             v=[ops.adamw_state(tiny, bits=8)[1]], master=[None])
    call(x, 1, beta1=0.0)
    m = x["m"][0].dequantize()
    assert x["m"][0].scale[1].item() == 0 and (m[128:] <= 2.0 ** -127 * 2.0 ** -6).all()
    assert ((m[:128].double() / 3e38 - 1).abs() <= 2.0 ** -3).all()


def test_moments_in_8_bits_are_the_float32_steps_rounded_once():
    """Every float32 step of m, v and the root is the correctly rounded one
    (torch's products, sums and roots on this device), so that each code and
    scale is exactly the rounding of it: 2^20 gradients from 2^-40 to 2^40, some
    chosen so that both terms of m cancel."""
    n, t, beta1, beta2 = 1 << 20, 12, 0.9, 0.999
    g = gen(16)
    x = lists([n], F32, BF16, False, 8, 16)
    size = torch.exp2(torch.randint(-40, 41, (n // 128,), generator=g, device="cuda").float()).repeat_interleave(128)
    x["g"][0].copy_(x["g"][0].float() * size)
    old = x["m"][0].dequantize()
    x["g"][0][:: 7] = (-9.0 * old[:: 7]).to(BF16)
    root = x["v"][0].dequantize()
    grad = x["g"][0].float()
    call(x, t, beta1=beta1, beta2=beta2)
    m = beta1 * old + (1 - beta1) * grad
    v = beta2 * (root * root) + (1 - beta2) * grad * grad
    part = torch.from_numpy((ref.words(0, n, t, SEED) & 0xFFFF) * 16 + 8).cuda()
    assert (m == 0).sum() > 100
    for name, want in (("m", m), ("v", v.sqrt())):
        top, k = torch.frexp(want.view(-1, 128).abs().amax(1))
        e = (k - 9 + (top > 0.875).int()).repeat_interleave(128)
        bits = torch.ldexp(want, -e - 120).view(torch.int32).long() & 0xFFFFFFFF
        code = (((bits & 0x7FFFFFFF) + part) >> 20) | (bits >> 24 & 0x80)
        if name == "v":
            code = torch.where((want > 0) & (code == 0), 1, code)
        got = x[name][0]
        assert torch.equal(got.scale.int(), e[::128] + 127), name
        assert torch.equal(got.data.view(torch.uint8).long(), code), name


def test_random_rounding_keeps_the_average():
    """600 steps without gradients: v falls by beta2 each, its root by 0.26 in
    all, in steps of 0.0005 of it, where the nearest E4M3 number is itself.  The
    mean over 2^16 elements is the exact one within its spread: a rounding adds
    at most 1/4 step^2, (2^-3)^2 / 4 of the root squared, and 600 of them act
    on a sum."""
    n, t = 1 << 16, 600
    p = torch.zeros(n, device="cuda")
    m, v = ops.adamw_state(p, bits=8)
    root = 0.5 + torch.rand(n, generator=gen(14), device="cuda")
    v.scale.fill_(127 - 8)
    v.data.copy_((root * 256).to(E4))
    first = v.dequantize().double().mean().item()
    g = torch.zeros(n, device="cuda")
    for k in range(1, t + 1):
        ops.adamw([p], [g], [m], [v], k, lr=0.0, beta2=0.999, seed=SEED)
    want = first * 0.999 ** (t / 2)
    got = v.dequantize().double().mean().item()
    # a walk's steps are probabilities q of about 0.0005 / step: variance q step^2 each
    spread = (t * 0.0005 * 0.125) ** 0.5 / n ** 0.5
    assert abs(got / want - 1) <= 6 * spread


def test_random_rounding_of_bfloat16():
    """The mean of the rounded parameters is the float32 one: 2^20 of them, each off by at most a step of 2^-7."""
    n = 1 << 20
    p = torch.full((n,), 1.0, device="cuda").bfloat16()
    m, v = torch.full((n,), 1e-3, device="cuda"), torch.full((n,), 1e-6, device="cuda")
    ops.adamw([p], [torch.full((n,), 1e-3, device="cuda")], [m], [v], 100000, lr=1e-3, seed=SEED)
    # p = 1 - 1e-3 (m / sqrt(v) = 1): between 1 - 2^-8 and 1, a share 0.001 / 2^-8 goes down
    share = (p.float() < 1).double().mean().item()
    q = 1e-3 * 256
    assert abs(share - q) <= 6 * (q * (1 - q) / n) ** 0.5 + 1e-4
    assert set(p.float().unique().tolist()) == {1.0, 1 - 2.0 ** -8}


@pytest.mark.parametrize("sizes", [[], [0], [1], [7, 0, 8192, 8193], [1 << 20, 3], [33] * 2500])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_gradient_norm(sizes, dtype):
    """Squares of positive terms: the chain of a thread's sums (at most 8192 elements of a chunk over 256 threads, a
    thousandth of all chunks) and 40 more."""
    g = gen(sum(sizes) % 1000)
    ts = [torch.randn(n, generator=g, device="cuda").to(dtype) for n in sizes]
    got = ops.gradient_norm(ts)
    want = sum(t.double().square().sum().item() for t in ts) ** 0.5
    assert got.shape == () and got.dtype == F32 and abs(got.item() - want) <= 120 * E * want
    assert torch.equal(got, ops.gradient_norm(ts))
    if sizes and max(sizes) > 1:
        odd = [shifted(t, 1) for t in ts]
        assert abs(ops.gradient_norm(odd).item() - want) <= 120 * E * want


def test_gradient_norm_of_mixed_and_special():
    a, b, c = (torch.full((n,), 2.0, device="cuda", dtype=t) for n, t in ((100, F32), (50, F16), (25, BF16)))
    assert ops.gradient_norm([a, b, c]).item() == pytest.approx(700 ** 0.5, rel=1e-6)
    assert ops.gradient_norm([a.view(10, 10), b]).item() == pytest.approx(600 ** 0.5, rel=1e-6)
    assert ops.gradient_norm([a, a]).item() == pytest.approx(800 ** 0.5, rel=1e-6)
    a[3] = float("nan")
    assert torch.isnan(ops.gradient_norm([b, a]))
    a[3] = float("inf")
    assert ops.gradient_norm([b, a]).item() == float("inf")


def test_past_2_31_elements():
    n = (1 << 31) + 5000
    x = dict(p=[torch.ones(n, dtype=BF16, device="cuda")], g=[torch.full((n,), 1e-3, dtype=BF16, device="cuda")],
             m=[], v=[], master=[None])
    for k in (0, 1):
        x["mv"[k]].append(ops.adamw_state(x["p"][0], bits=8)[k])
    norm = ops.gradient_norm(x["g"])
    exact = float(x["g"][0][0].double()) * n ** 0.5
    assert abs(norm.item() - exact) <= 3e-5 * exact  # (chains of 2^31 / (1024 * 256 * 16) terms, and their pairs)
    call(x, 5)
    part = slice(n - 5000 - 200, n)  # across the border, at the end
    y = dict(p=[x["p"][0][part].clone().fill_(1)], g=[x["g"][0][part].clone()], m=[], v=[], master=[None])
    w = ref.words(n - 5200 - (n - 5200) % 128, 5400, 5, SEED)[(n - 5200) % 128:][:5200]
    p, nm, nv = ref.step(f64(y["p"][0]), f64(y["g"][0]), 0.0, 0.0, 5, HYPER["lr"], HYPER["beta1"], HYPER["beta2"],
                         HYPER["eps"], HYPER["weight_decay"])
    on_grid(f64(x["p"][0][part]), p, 20 * E * np.abs(p), ref.grid(p, np.zeros(5200), 7, -126), (w >> 16) / 65536, "p")
    m = x["m"][0]
    e = m.scale.float().cpu().numpy()[-1] - 127.0
    m_part = m.data[part].float().double().cpu().numpy() * 2.0 ** e
    on_grid(m_part, nm, 8 * E * nm, ref.grid(nm, np.full(5200, e), 3, -6), ((w & 0xFFFF) + 0.5) / 65536, "m")
    del x
    torch.cuda.empty_cache()


def test_streams_and_graphs():
    """Captured with its step on the device, replayed: the same bits as eager steps."""
    params = [torch.randn(n, generator=gen(n), device="cuda") for n in (5000, 129)]
    low = [p.bfloat16() for p in params]
    grads = [torch.randn(n, generator=gen(n + 1), device="cuda") * 1e-2 for n in (5000, 129)]

    def make():
        return (AdamW([p.clone() for p in params], lr=torch.full((), 1e-3, device="cuda"), captured=True),
                AdamW([p.clone() for p in low], lr=1e-3, bits=8, seed=3, captured=True))

    def step(pair, stream=None):
        norm = ops.gradient_norm(grads, stream=stream)
        for o in pair:
            o.step(grads, norm=norm, max_norm=0.5, stream=stream)

    eager, graphed, aside = make(), make(), make()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for k in range(4):
        for i, g in enumerate(grads):
            g.copy_(torch.randn(g.shape, generator=gen(100 * k + i), device="cuda"))
        s.wait_stream(torch.cuda.current_stream())
        step(eager)
        graph.replay()
        step(aside, s)
        torch.cuda.current_stream().wait_stream(s)
    assert eager[0].count.item() == 4
    for other in (graphed, aside):
        for a, b in zip(eager, other):
            assert torch.equal(a.count, b.count) and all(torch.equal(p, q) for p, q in zip(a.params, b.params))
            for i in range(2):
                assert all(torch.equal(p, q) for p, q in zip(a.moments(i), b.moments(i)))


def test_lists_that_can_be_read_once():
    """Generators, on the current stream and on another one."""
    x = lists([500, 70], BF16, F32, True, 8, 15)
    want, norm = cloned(x), ops.gradient_norm(x["g"])
    call(want, 3)
    s = torch.cuda.Stream()
    for stream in (None, s):
        y = cloned(x)
        s.wait_stream(torch.cuda.current_stream())
        assert torch.equal(ops.gradient_norm((g for g in x["g"]), stream=stream), norm)
        ops.adamw(iter(y["p"]), iter(y["g"]), iter(y["m"]), iter(y["v"]), 3, masters=iter(y["master"]), seed=SEED,
                  stream=stream, **HYPER)
        torch.cuda.current_stream().wait_stream(s)
        assert same(y, want) and not torch.equal(y["p"][0], x["p"][0])


def test_optimizer_object():
    p = [torch.randn(7, 33, generator=gen(1), device="cuda"), torch.randn(50, generator=gen(2), device="cuda").half()]
    opt = AdamW([t.clone() for t in p], lr=1e-2, weight_decay=0.1)
    x = dict(p=[t.clone() for t in p], g=[torch.randn_like(t) for t in p], master=[None, p[1].float()],
             m=[ops.adamw_state(t)[0] for t in p], v=[ops.adamw_state(t)[1] for t in p])
    for t in (1, 2, 3):
        opt.step(x["g"])
        ops.adamw(x["p"], x["g"], x["m"], x["v"], t, lr=1e-2, weight_decay=0.1, masters=x["master"])
    assert opt.count == 3 and all(torch.equal(a, b) for a, b in zip(opt.params, x["p"]))
    assert torch.equal(opt.moments(0)[1], x["v"][0]) and torch.equal(opt.masters[1], x["master"][1])


def test_refusals():
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    m, v = ops.adamw_state(p)
    m8, v8 = ops.adamw_state(p, bits=8)
    h = p.half()

    def adamw(params=None, grads=None, ms=None, vs=None, step=1, **kw):
        ops.adamw([p] if params is None else params, [g] if grads is None else grads, [m] if ms is None else ms,
                  [v] if vs is None else vs, step, **dict(dict(lr=1e-3), **kw))

    one = torch.ones(1, device="cuda")
    for bad in (dict(params=[p.double()]), dict(params=[p.cpu()]), dict(params=[p, p]), dict(grads=[g[:32]]),
                dict(grads=[g.view(8, 8)]), dict(params=[torch.zeros(128, device="cuda")[::2]]), dict(grads=[g.int()]),
                dict(grads=[None]), dict(ms=[None]), dict(ms=[m8]), dict(vs=[v8]), dict(ms=[m.half()]),
                dict(ms=[ops.Fp8Vector(m8.data, m8.scale.int())], vs=[v8]),
                dict(ms=[ops.Fp8Vector(m8.data, v8.scale[:0])], vs=[v8]), dict(ms=[v]), dict(vs=[p]),
                dict(ms=[ops.Fp8Vector(v8.data, m8.scale)], vs=[v8]),
                dict(masters=[one]), dict(masters=[p.clone()]), dict(params=[h]), dict(params=[h], masters=[None]),
                dict(params=[h], masters=[h]), dict(masters=[]) | dict(params=[h]), dict(step=0), dict(step=-1),
                dict(step=one), dict(step=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(step=torch.ones(1, dtype=torch.int64)), dict(lr=-1.0), dict(lr=float("nan")), dict(lr=one.double()),
                dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=-1e-8), dict(weight_decay=-0.1),
                dict(norm=one.cpu()), dict(norm=one.half()), dict(norm=one, max_norm=0.0),
                dict(norm=one, max_norm=float("nan")), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(seed=-1), dict(seed=1 << 64)):
        with pytest.raises((ValueError, B.RotError, TypeError)):
            adamw(**bad)
    x, y = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    with pytest.raises((ValueError, B.RotError)):  # a parameter twice
        ops.adamw([p, p], [g, g], [m, x], [v, y], 1, lr=1e-3)
    for bad in ([g.cpu()], [g.int()], [torch.zeros(8, 8, device="cuda").t()[:, :4]], [None]):
        with pytest.raises((ValueError, B.RotError)):
            ops.gradient_norm(bad)
    with pytest.raises(ValueError):
        ops.adamw_state(p, bits=4)


def test_the_operators_together():
    """A layer's step: norm, fused projection in 8 bits, norm of the heads with the rotation, attention, loss; back
    through all of it; clipping over all gradients; the matrix by RotatedAdam, the vectors by AdamW.  The heads'
    gradients against autograd's in 64 bits, the update against the formulas."""
    g = gen(21)
    tokens, width, q_heads, k_heads, dim = 48, 128, 4, 2, 32
    x = torch.randn(tokens, width, generator=g, device="cuda")
    w = torch.randn((q_heads + 2 * k_heads) * dim, width, generator=g, device="cuda") * width ** -0.5
    vectors = [torch.ones(width, device="cuda"), torch.ones(dim, device="cuda"), torch.ones(dim, device="cuda")]
    rotary = ops.rotary_table(ops.rotary_frequencies(dim))
    at = torch.cat([torch.arange(20), torch.arange(28)]).cuda()  # two sequences
    inside = torch.block_diag(torch.ones(20, 20), torch.ones(28, 28)).cuda().tril() > 0
    aim = torch.randn(tokens, q_heads * dim, generator=g, device="cuda") / tokens

    def attend(q, k, v):
        k, v = (t.repeat_interleave(q_heads // k_heads, 1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q, k) * dim ** -0.5
        return torch.einsum("hqk,khd->qhd", s.masked_fill(~inside, float("-inf")).softmax(-1), v).flatten(1)

    opt = RotatedAdam([tuple(w.shape)], 64 << 20, lr=1e-3)
    rest = AdamW(vectors, lr=1e-2)
    for step in range(1, 4):
        quantized, transposed = ops.fp8_quantize(w, block_rows=128, transposed=True)
        y, h, mean, rstd = ops.layer_norm(x, vectors[0])
        qkv = ops.fp8_linear(y, quantized).view(tokens, -1, dim)
        q, k, v = qkv.split([q_heads, k_heads, k_heads], 1)
        qn, kn = ops.head_norm(q, vectors[1], k, vectors[2], rotary=rotary, positions=at)
        # attention's own backward pass in torch, on the operators' results
        leaves = [t.clone().requires_grad_() for t in (qn, kn, v)]
        (attend(*leaves) * aim).sum().backward()
        dqn, dkn, dv = (t.grad for t in leaves)
        dqkv = torch.empty_like(qkv)
        _, _, dwq, dwk = ops.head_norm_backward(dqn, q, vectors[1], dkn, k, vectors[2], rotary=rotary, positions=at,
                                                out=dqkv[:, :q_heads], k_out=dqkv[:, q_heads:q_heads + k_heads])
        dqkv[:, q_heads + k_heads:] = dv
        dy, dw = ops.fp8_linear_backward(dqkv.flatten(1), y, transposed)
        _, _, dg, _ = ops.layer_norm_backward(dy, h, mean, rstd, vectors[0], bias=False)
        # the same from the heads' inputs on, by autograd in 64 bits
        deep = [t.detach().double().requires_grad_() for t in (q, k, v, vectors[1], vectors[2])]
        turned = []
        for t, u in ((deep[0], deep[3]), (deep[1], deep[4])):
            t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * u
            a = ref.angles(rotary.turns, at)[:, None]
            n = dim // 2
            turned.append(torch.cat([t[..., :n] * a.cos() - t[..., n:] * a.sin(),
                                     t[..., n:] * a.cos() + t[..., :n] * a.sin()], -1))
        (attend(*turned, deep[2]) * aim.double()).sum().backward()
        for got, want in ((dqkv[:, :q_heads], deep[0]), (dqkv[:, q_heads:q_heads + k_heads], deep[1]),
                          (dv, deep[2]), (dwq, deep[3]), (dwk, deep[4])):
            # (attention in float32: sums of 48 and 32 terms, exponentials; 200 E of the gradient's size)
            assert ((got.double() - want.grad).norm() <= 200 * E * want.grad.norm()).item()
        grads = [dg, dwq, dwk]
        norm = ops.gradient_norm([dw, *grads])
        total = sum(t.double().square().sum() for t in (dw, *grads)).sqrt()
        assert abs(norm.item() / total.item() - 1) <= 64 * E
        before, moments = [p.double().cpu().numpy() for p in vectors], [rest.moments(i) for i in range(3)]
        rest.step(grads, norm=norm, max_norm=0.5 * norm.item())
        opt.step([w], [dw * 0.5], refresh=step == 2)
        for i in range(3):
            want, _, _ = ref.step(before[i], f64(grads[i]), f64(moments[i][0]), f64(moments[i][1]), step, 1e-2, 0.9,
                                  0.999, 1e-8, 0.0, 0.5)
            assert np.abs(f64(vectors[i]) - want).max() <= 64 * E
    assert opt.status() == B.ROT_OK and ops.status() == B.ROT_OK
