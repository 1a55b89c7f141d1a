"""The heads' entry to attention and the step of the parameters next to the matrices, as measured cases.

Rotary positions (`rotate`) and the norm of queries and keys for each head with the rotation in the same pass
(`heads`), forward and backward; AdamW over many tensors at once (`adamw`), its states in 32 or in 8 bits, with the
norm of the whole gradient to clip by.  `run` computes a case in elementary torch operations (`own` false) or through
the framework's entry points (`own` true); `exact` restates it in 64 bits.
"""

import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.1
LOW = 0xFFFFFFFF


def _heads(op, backward, batch, tokens, q, k, dim, rotated, kind, **more):
    return {"op": op, "backward": backward, "batch": batch, "tokens": tokens, "q_heads": q, "k_heads": k, "dim": dim,
            "rotated": rotated, "type": kind, "interleaved": False, "fused": False, "packed": False, "first": 0,
            "factor": 1.0, "magnitude": 1.0, **more}


def _adamw(layout, count, largest, param, grad, master, bits, clip, draw=0):
    return {"op": "adamw", "layout": layout, "count": count, "largest": largest, "param": param, "grad": grad,
            "master": master, "bits": bits, "clip": clip, "draw": draw}


def listed():
    return [
        # a new token for each of 8 long sequences: 16 query and 8 key heads of 128
        {"name": "rotate_token", **_heads("rotate", False, 8, 1, 16, 8, 128, 128, "bf16", first=100000)},
        # a training step's 16384 tokens, packed sequences, queries and keys as they lie in the fused projection
        {"name": "rotate_block", **_heads("rotate", False, 4, 4096, 16, 8, 128, 128, "bf16", fused=True, packed=True)},
        # the gradient through neighbouring pairs of two thirds of the head, far out under frequencies scaled by 8
        {"name": "rotate_long_grad", **_heads("rotate", True, 1, 4099, 12, 3, 96, 64, "f16", interleaved=True,
                                              first=120000, factor=8.0, magnitude=1.2)},
        # one new token: norm of its heads and rotation, latency alone
        {"name": "heads_token", **_heads("heads", False, 1, 1, 16, 8, 128, 128, "bf16", first=4000)},
        # the entry to attention of a training step
        {"name": "heads_block", **_heads("heads", False, 4, 4096, 16, 8, 128, 128, "bf16", fused=True, packed=True)},
        # its backward pass, with the gradients of both weights
        {"name": "heads_block_grad", **_heads("heads", True, 4, 4096, 16, 8, 128, 128, "bf16", fused=True, packed=True)},
        # a small float32 model whose heads have an odd width, a part of them rotated
        {"name": "heads_odd_grad", **_heads("heads", True, 3, 335, 5, 5, 75, 38, "f32", interleaved=True)},
        # wide heads that share one key head
        {"name": "heads_wide", **_heads("heads", False, 2, 2049, 8, 1, 256, 128, "f16")},
        # the vectors of 28 blocks and the last norm: 113 small tensors
        {"name": "adamw_vectors", **_adamw("vectors", 28, 0, "f32", "f32", False, 32, False)},
        # the matrices of 7 blocks in float32, with clipping
        {"name": "adamw_blocks", **_adamw("blocks", 7, 0, "f32", "f32", False, 32, True)},
        # the same in bfloat16 without a float32 copy, states in 8 bits
        {"name": "adamw_blocks_8bit", **_adamw("blocks", 7, 0, "bf16", "bf16", False, 8, False)},
        # an embedding of 100277 x 2048 and the vectors, bfloat16 with float32 copies, states in 8 bits, clipping
        {"name": "adamw_embedding_8bit", **_adamw("embedding", 28, 0, "bf16", "bf16", True, 8, True)},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm; about half of them odd."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rotate", "heads", "heads", "adamw", "adamw"])
    if op == "adamw":
        param, master = rng.choice([("f32", False), ("bf16", False), ("bf16", True), ("f16", True)])
        count = _spread(rng, 1, 300)
        grad = rng.choice([param, param, "f32"])
        return _adamw("drawn", count, _spread(rng, 10, 150_000_000 // count), param, grad, master, rng.choice([32, 8]),
                      rng.random() < 0.5, rng.randrange(1 << 20))
    # widths of whole 16-byte runs, and any other
    dim = 8 * rng.randint(2, 32) if rng.random() < 0.6 else _spread(rng, 6, 300)
    rotated = rng.choice([dim, dim, dim // 2]) // 2 * 2
    q = _spread(rng, 1, 40)
    k = max(1, q // rng.choice([1, 2, 4, 8]))
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    total = _spread(rng, 1, min(32768, (25_000_000 if kind == "f32" else 50_000_000) // ((q + k) * dim)))
    batch = min(total, rng.choice([1, 1, 2, 3, 8]))
    return _heads(op, rng.random() < 0.5, batch, total // batch, q, k, dim, rotated, kind,
                  interleaved=rng.random() < 0.4, fused=rng.random() < 0.5, packed=rng.random() < 0.5,
                  first=rng.choice([0, 0, 1000, 1_000_000]), factor=rng.choice([1.0, 1.0, 4.0, 32.0]),
                  magnitude=rng.choice([1.0, 1.0, 1.35]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _frequencies(rotated, factor, base=1e6, length=8192.0):
    """Radians a position adds for each pair.  A factor slows the pairs that do not complete a turn over the original
    length by it, leaves those of 4 turns and more, and blends in between."""
    f = base ** (-torch.arange(0, rotated, 2, dtype=torch.float64, device="cuda") / max(rotated, 1))
    kept = ((f * length / (2 * math.pi) - 1) / 3).clamp(0, 1)
    return f * (kept + (1 - kept) / factor)


def _shapes(case):
    n, layout = case["count"], case["layout"]
    if layout == "drawn":
        r = random.Random(case["draw"])
        return [(_spread(r, 1, case["largest"]),) for _ in range(n)]
    if layout == "blocks":
        return [(2048, 2048), (1024, 2048), (1024, 2048), (2048, 2048), (6144, 2048), (6144, 2048), (2048, 6144)] * n
    vectors = [(2048,), (2048,), (128,), (128,)] * n + [(2048,)]
    return ([(100277, 2048)] if layout == "embedding" else []) + vectors


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    if case["op"] == "adamw":
        return _prepare_adamw(s, case, seed, g)
    B, S, q, k, D = (case[n] for n in ("batch", "tokens", "q_heads", "k_heads", "dim"))
    dtype = TYPES[case["type"]]

    def heads(scale, fused):
        # queries, keys and values of one projection, or tensors of their own; a few channels much larger than the rest
        x = torch.randn(B, S, q + k * (2 if fused else 1), D, generator=g, device="cuda").mul_(scale)
        x[..., torch.randperm(D, generator=g, device="cuda")[:max(1, D // 64)]] *= 8.0
        x = x.to(dtype)
        a, b = x[:, :, :q], x[:, :, q:q + k]
        return (a, b) if fused else (a.contiguous(), b.contiguous())

    s["q"], s["k"] = heads(1.0, case["fused"])
    if case["backward"]:
        s["dq"], s["dk"] = heads(1e-3, False)
    if case["op"] == "heads":
        s["wq"], s["wk"] = (1.0 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    at = torch.arange(S, device="cuda").expand(B, S)
    if case["packed"]:  # several sequences behind one another: positions begin again
        start = torch.rand(B, S, generator=g, device="cuda") < 4.0 / S
        at = at - torch.cummax(torch.where(start, at, 0), 1).values
    far = torch.randint(1 + case["first"] // 8, (B, 1), generator=g, device="cuda")
    s["positions"] = (at + case["first"] + far).contiguous()
    s["frequencies"] = _frequencies(case["rotated"], case["factor"])
    # the part of a turn that a position adds, in units of 2^-64
    s["turns"] = (s["frequencies"] / (2 * math.pi) * 2.0 ** 64).round().to(torch.int64)
    return s


def _prepare_adamw(s, case, seed, g):
    shapes = _shapes(case)
    sizes = [math.prod(x) for x in shapes]
    # every tensor at a multiple of 128 elements of one buffer for each kind, the rest zeros
    starts, n = [], 0
    for size in sizes:
        starts.append(n)
        n += -(-size // 128) * 128
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    for at, size in zip(starts, sizes):
        used[at:at + size] = True

    def normal(std):
        return torch.randn(n, generator=g, device="cuda").mul_(std).mul_(used)

    def views(flat):
        return [flat[at:at + size].view(shape) for at, size, shape in zip(starts, sizes, shapes)]

    # gradients that differ in size from place to place
    s["g"] = (normal(1e-3) * torch.exp(normal(1.0))).to(TYPES[case["grad"]])
    w = normal(0.02)
    s["p"] = w.to(TYPES[case["param"]])
    s["master"] = w if case["master"] else None
    m, r = normal(3e-4), normal(1e-3).abs_().add_(1e-4).mul_(used)
    if case["bits"] == 32:
        s["m"], s["v"] = m, r.square_()
    else:
        half = torch.full((n,), 0x8000, dtype=torch.int32, device="cuda")
        s["m"], s["m_scale"] = _rounded8(m, half)
        s["v"], s["v_scale"] = _rounded8(r, half)
    for name in ("g", "p", "master", "m", "v"):
        s[name + "_list"] = views(s[name]) if s[name] is not None else None
    for name in ("m", "v"):
        if case["bits"] == 8:
            s[name + "_scale_list"] = [s[name + "_scale"][at // 128:at // 128 + -(-size // 128)]
                                       for at, size in zip(starts, sizes)]
    s["step"], s["seed"] = 100 + seed % 1000, 0x9E3779B97F4A7C15 ^ (seed * 0x2545F4914F6CDD1D & (1 << 64) - 1)
    s["max_norm"] = 1.0
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _angles(s):
    """Cosine and sine for each token and pair; 64 bits, since a far position's angle has many turns."""
    angle = s["positions"].double()[..., None] * s["frequencies"]
    m = s["case"]["magnitude"]
    return (angle.cos() * m).float()[:, :, None], (angle.sin() * m).float()[:, :, None]


def _rotate(x, cos, sin, interleaved):
    n = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _norm_heads(x, w):
    f = x.float()
    return f / torch.sqrt(f.square().mean(-1, keepdim=True) + EPS) * w


def _norm_heads_grad(g, x, w):
    f = x.float()
    rstd = 1.0 / torch.sqrt(f.square().mean(-1, keepdim=True) + EPS)
    hat, gw = f * rstd, g * w
    dx = rstd * (gw - hat * (gw * hat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * hat).sum((0, 1, 2))


def _words(n, offset, seed):
    """The generator's 32-bit words 0 .. n - 1 (n a multiple of 4): Philox4x32-10 at the counters (i div 4, offset)
    under the key `seed` (Salmon, Moraes, Dror and Shaw, SC 2011)."""
    j = torch.arange(n // 4, dtype=torch.int64, device="cuda")
    c = [j & LOW, j >> 32, torch.full_like(j, offset & LOW), torch.full_like(j, offset >> 32 & LOW)]
    k0, k1 = seed & LOW, seed >> 32 & LOW
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32 & LOW) ^ c[1] ^ k0, b & LOW, (a >> 32 & LOW) ^ c[3] ^ k1, a & LOW]
        k0, k1 = k0 + 0x9E3779B9 & LOW, k1 + 0xBB67AE85 & LOW
    return torch.stack(c, 1).view(-1)


def _rounded8(x, random16):
    """x in e4m3 and a byte e for each 128 elements, their scale 2^(e - 127): the least with all of them within 448 of
    it.  Rounded up where the part cut off and (16 random bits + 1/2) / 2^16 come to one step; e4m3's bits are the
    upper ones of a float32 of 2^-120 times the value."""
    top, k = torch.frexp(x.view(-1, 128).abs().amax(1))
    e = torch.where(top > 0, k - 9 + (top > 0.875).to(torch.int32), -127).clamp(min=-127)
    scaled = (x.view(-1, 128) * (127 - e << 23).view(torch.float32)[:, None] * 2.0 ** -120).view(-1)
    bits = scaled.view(torch.int32)
    q = ((bits & 0x7FFFFFFF) + (random16 << 4) + 8 >> 20) | (bits >> 24 & 0x80)
    return q.to(torch.uint8).view(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _values8(q, scale):
    two = torch.where(scale > 0, scale.to(torch.int32) << 23, 1 << 22).view(torch.float32)
    return (q.float().view(-1, 128) * two[:, None]).view(-1)


def _plain_adamw(s):
    c, t = s["case"], s["step"]
    g, norm = s["g"].float(), None
    if c["clip"]:
        norm = g.square().sum(dtype=torch.float64).sqrt().float()
        g = g * torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0)
    eight, rounds = c["bits"] == 8, c["param"] == "bf16" and not c["master"]
    if eight or rounds:
        words = _words(g.numel(), t, s["seed"])
        low, high = (words & 0xFFFF).to(torch.int32), (words >> 16).to(torch.int32)
    if eight:
        m, v = _values8(s["m"], s["m_scale"]), _values8(s["v"], s["v_scale"]).square()
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    r = v.sqrt()
    p = (s["master"] if c["master"] else s["p"]).float()
    p = p * (1 - LR * DECAY) - LR / (1 - BETA1 ** t) * m / (r / math.sqrt(1 - BETA2 ** t) + ADAM_EPS)
    if eight:
        q, e = _rounded8(m, low)
        s["m"].copy_(q), s["m_scale"].copy_(e)
        q, e = _rounded8(r, low)
        # a root that is not zero does not become zero
        q = torch.where((r > 0) & (q.view(torch.uint8) == 0), 1, q.view(torch.uint8)).view(torch.float8_e4m3fn)
        s["v"].copy_(q), s["v_scale"].copy_(e)
    else:
        s["m"].copy_(m), s["v"].copy_(v)
    if c["master"]:
        s["master"].copy_(p), s["p"].copy_(p)
    elif rounds:
        s["p"].copy_((p.view(torch.int32) + high & ~0xFFFF).view(torch.float32))
    else:
        s["p"].copy_(p)
    return norm


def _run_adamw(s):
    c = s["case"]
    s["step"] += 1
    if own:
        from matrix_optimizer_step_rot_gb300 import operators as ops
        m, v = s["m_list"], s["v_list"]
        if c["bits"] == 8:
            m = [ops.Fp8Vector(*x) for x in zip(m, s["m_scale_list"])]
            v = [ops.Fp8Vector(*x) for x in zip(v, s["v_scale_list"])]
        norm = ops.gradient_norm(s["g_list"]) if c["clip"] else None
        ops.adamw(s["p_list"], s["g_list"], m, v, s["step"], lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS,
                  weight_decay=DECAY, masters=s["master_list"], norm=norm, max_norm=s["max_norm"], seed=s["seed"])
    else:
        norm = _plain_adamw(s)
    out = {"p": s["p"], "m": s["m"], "v": s["v"]}
    if c["bits"] == 8:  # the states' values: e4m3 numbers and the powers of two over them
        out |= {n + "_scale": s[n + "_scale"].view(torch.float8_e8m0fnu) for n in ("m", "v")}
    if c["master"]:
        out["master"] = s["master"]
    if norm is not None:
        out["norm"] = norm
    return out


def run(state):
    s, c = state, state["case"]
    if c["op"] == "adamw":
        return _run_adamw(s)
    if own:
        from matrix_optimizer_step_rot_gb300 import operators as ops
        rotary = ops.Rotary(s["turns"], c["magnitude"], c["interleaved"])
    if c["op"] == "rotate":
        a, b = (s["dq"], s["dk"]) if c["backward"] else (s["q"], s["k"])
        if own:
            a, b = (ops.rotate_backward if c["backward"] else ops.rotate)(a, rotary, b, positions=s["positions"])
        else:
            cos, sin = _angles(s)
            sin = -sin if c["backward"] else sin
            a, b = (_rotate(x.float(), cos, sin, c["interleaved"]).to(x.dtype) for x in (a, b))
        return {"q": a, "k": b}
    if own:
        if not c["backward"]:
            a, b = ops.head_norm(s["q"], s["wq"], s["k"], s["wk"], EPS, rotary=rotary, positions=s["positions"])
            return {"q": a, "k": b}
        dq, dk, dwq, dwk = ops.head_norm_backward(s["dq"], s["q"], s["wq"], s["dk"], s["k"], s["wk"], EPS,
                                                  rotary=rotary, positions=s["positions"])
        return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}
    cos, sin = _angles(s)
    if not c["backward"]:
        a, b = (_rotate(_norm_heads(x, w), cos, sin, c["interleaved"]).to(x.dtype)
                for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
        return {"q": a, "k": b}
    (dq, dwq), (dk, dwk) = (_norm_heads_grad(_rotate(d.float(), cos, -sin, c["interleaved"]), x, w)
                            for d, x, w in ((s["dq"], s["q"], s["wq"]), (s["dk"], s["k"], s["wk"])))
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def work(case):
    c = case
    if c["op"] == "adamw":
        n = sum(math.prod(x) for x in _shapes(c))
        p, g = BYTES[c["param"]], BYTES[c["grad"]]
        each = (8 + p if c["master"] else 2 * p) + g * (2 if c["clip"] else 1) + (16 if c["bits"] == 32 else 4 + 4 / 128)
        return {"bytes": int(n * each), "flops": (16 + 2 * c["clip"]) * n}
    n = c["batch"] * c["tokens"] * (c["q_heads"] + c["k_heads"]) * c["dim"]
    arrays = 3 if c["op"] == "heads" and c["backward"] else 2
    return {"bytes": n * arrays * BYTES[c["type"]] + 8 * c["batch"] * c["tokens"],
            "flops": n * {"rotate": 3, "heads": 15 if c["backward"] else 7}[c["op"]]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_turned(x, s, sign):
    """Pairs as complex numbers times magnitude e^(+-i angle)."""
    c, h = s["case"], s["case"]["rotated"] // 2
    phase = torch.einsum("bs,i->bsi", s["positions"].double(), s["frequencies"]) * sign
    unit = torch.polar(torch.full_like(phase, c["magnitude"]), phase).unsqueeze(2)
    part = x[..., :2 * h].double()
    if c["interleaved"]:
        z = torch.view_as_complex(part.unflatten(-1, (h, 2)).contiguous()) * unit
        part = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(part[..., :h], part[..., h:]) * unit
        part = torch.cat((z.real, z.imag), -1)
    return torch.cat((part, x[..., 2 * h:].double()), -1)


def _exact_words(n, offset, seed):
    """The generator's words by whole numbers in 16-bit halves."""
    def product(x, m):
        x0, x1, m0, m1 = x & 0xFFFF, x >> 16, m & 0xFFFF, m >> 16
        mid = x1 * m0 + (x0 * m0 >> 16)
        low = x0 * m1 + (mid & 0xFFFF)
        return x1 * m1 + (mid >> 16) + (low >> 16), (low & 0xFFFF) << 16 | x0 * m0 & 0xFFFF

    i = torch.arange(n // 4, device="cuda")
    w0, w1 = i % 2 ** 32, i // 2 ** 32
    w2, w3 = torch.zeros_like(i) + offset % 2 ** 32, torch.zeros_like(i) + offset // 2 ** 32
    for r in range(10):
        key0, key1 = (seed + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        hi0, lo0 = product(w0, 0xD2511F53)
        hi2, lo2 = product(w2, 0xCD9E8D57)
        w0, w1, w2, w3 = hi2 ^ w1 ^ key0, lo2, hi0 ^ w3 ^ key1, lo0
    out = torch.empty(n // 4, 4, dtype=torch.int64, device="cuda")
    for k, w in enumerate((w0, w1, w2, w3)):
        out[:, k] = w
    return out.flatten()


def _exact_up(x, bits, least, part):
    """|x| on the grid of `bits` fraction bits, exponents from `least` up: to the step below, or the one above where the
    rest and `part` come to a step."""
    size = x.abs()
    e = torch.frexp(size).exponent - 1
    step = torch.ldexp(torch.ones_like(size), e.clamp(min=least) - bits)
    return torch.copysign(torch.floor(size / step + part) * step, x)


def _exact_state8(x, part, root):
    """(the e4m3 numbers, the scales) of x."""
    top = x.view(-1, 128).abs().amax(1)
    e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)), -127.0).clamp(min=-127)
    e = torch.where((e > -127) & (top <= 448.0 * torch.exp2(e - 1)), e - 1, e)  # the logarithm's rounding
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    scale = torch.exp2(e)
    y = _exact_up((x.view(-1, 128) / scale[:, None]).view(-1), 3, -6, part)
    if root:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
    return y, scale


def _exact_adamw(s):
    c, t = s["case"], s["step"] + 1
    g, out = s["g"].double(), {}
    if c["clip"]:
        out["norm"] = torch.linalg.vector_norm(g)
        g = g * min(1.0, s["max_norm"] / out["norm"].item())
    eight = c["bits"] == 8
    m, v = s["m"].double(), s["v"].double()
    if eight:
        m, v = ((x.view(-1, 128) * torch.exp2(e.double() - 127)[:, None]).view(-1)
                for x, e in ((m, s["m_scale"]), (v, s["v_scale"])))
        v = v ** 2
    m.lerp_(g, 1 - BETA1)
    v.lerp_(g ** 2, 1 - BETA2)
    p = (s["master"] if c["master"] else s["p"]).double()
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)) ** 0.5 + ADAM_EPS)
    words = _exact_words(g.numel(), t, s["seed"])
    if eight:
        part = ((words % 65536).double() + 0.5) / 65536
        m, out["m_scale"] = _exact_state8(m, part, False)
        v, out["v_scale"] = _exact_state8(v ** 0.5, part, True)
    if c["master"]:
        out["master"] = p
    elif c["param"] == "bf16":
        p = _exact_up(p, 7, -126, (words // 65536).double() / 65536)
    return out | {"p": p, "m": m, "v": v}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    if case["op"] == "rotate":
        a, b = (s["dq"], s["dk"]) if case["backward"] else (s["q"], s["k"])
        sign = -1.0 if case["backward"] else 1.0
        return {"q": _exact_turned(a, s, sign), "k": _exact_turned(b, s, sign)}
    out = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w" + n].double()
        scale = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / case["dim"] + EPS) ** -0.5
        if not case["backward"]:
            out[n] = _exact_turned(x * scale * w, s, 1.0)
            continue
        g = _exact_turned(s["d" + n], s, -1.0)
        along = torch.einsum("bshd,d,bshd->bsh", g, w, x)[..., None]
        out["d" + n] = g * w * scale - x * along * scale ** 3 / case["dim"]
        out["d" + n + "_weight"] = torch.einsum("bshd,bshd,bsh->d", g, x, scale[..., 0])
    return out
