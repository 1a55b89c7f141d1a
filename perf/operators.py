"""The training operators next to the optimizer step, as measured cases.

Layer norm with the residual stream and dropout before it (forward and backward), counter-based dropout, the
clipped policy loss with its gradient, and linear layers in 8-bit floating point with power-of-two block scales.
`run` computes a case in elementary torch operations (`own` false) or through the framework's entry points
(`own` true); `exact` restates it in 64 bits.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.05


def listed():
    return [
        # one token of a decoder block of width 2048: latency alone
        {"name": "norm_token", "op": "norm", "backward": False, "rows": 1, "cols": 2048, "pad": 0, "type": "bf16",
         "residual": True, "p": 0.0},
        # the block entry of a training step: 16384 tokens, width 4096, residual add and dropout in front of the norm
        {"name": "norm_block", "op": "norm", "backward": False, "rows": 16384, "cols": 4096, "pad": 0, "type": "bf16",
         "residual": True, "p": 0.1},
        # its backward pass at width 2048 over a batch whose last sequence is cut short
        {"name": "norm_block_grad", "op": "norm", "backward": True, "rows": 16383, "cols": 2048, "pad": 0,
         "type": "bf16", "residual": True, "p": 0.1},
        # a small float32 model of odd width, rows of a wider buffer, plain norm
        {"name": "norm_odd_grad", "op": "norm", "backward": True, "rows": 1000, "cols": 641, "pad": 7, "type": "f32",
         "residual": False, "p": 0.0},
        # dropout of the feed-forward activation of a training step (width 6144) with its residual
        {"name": "dropout_ffn", "op": "dropout", "backward": False, "rows": 16384, "cols": 6144, "pad": 0,
         "type": "bf16", "residual": True, "p": 0.1},
        # the gradient through a small odd-sized dropout
        {"name": "dropout_odd_grad", "op": "dropout", "backward": True, "rows": 777, "cols": 1001, "pad": 0,
         "type": "f32", "residual": False, "p": 0.25},
        # a handful of sampled tokens, float32 logits: loss and gradient
        {"name": "policy_few", "op": "policy", "grad": True, "tokens": 7, "vocab": 32768, "type": "f32", "masked": 0.0},
        # a policy step: prompt tokens masked, 65536 entries in the vocabulary
        {"name": "policy_step", "op": "policy", "grad": True, "tokens": 4096, "vocab": 65536, "type": "bf16",
         "masked": 0.2},
        # scoring: the log-probabilities that a policy step takes as its old and reference values, odd vocabulary
        {"name": "policy_score", "op": "policy", "grad": False, "tokens": 2049, "vocab": 100277, "type": "bf16",
         "masked": 0.0},
        # one token through a linear layer with weights kept in 8 bits: reading the weights
        {"name": "linear_token", "op": "linear", "backward": False, "tokens": 1, "inner": 2048, "outer": 6144,
         "type": "bf16"},
        # the up projection of a training step, 4096 to 12288
        {"name": "linear_up", "op": "linear", "backward": False, "tokens": 8192, "inner": 4096, "outer": 12288,
         "type": "bf16"},
        # both gradients of a 2048 to 6144 layer over a ragged batch, the weight's in float32 for the optimizer
        {"name": "linear_grad", "op": "linear", "backward": True, "tokens": 4099, "inner": 2048, "outer": 6144,
         "type": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm; about half of them odd."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "dropout", "policy", "linear"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm", "dropout"):
        cols = _spread(rng, 33, 12288)
        rows = _spread(rng, 1, max(1, 60_000_000 // cols if kind == "f32" else 100_000_000 // cols))
        return {"op": op, "backward": rng.random() < 0.5, "rows": min(rows, 32768), "cols": cols,
                "pad": rng.choice([0, 0, 0, 3, 8, 40]), "type": kind, "residual": rng.random() < 0.5,
                "p": rng.choice([0.0, 0.1, 0.25]) if op == "norm" else rng.choice([0.05, 0.1, 0.5])}
    if op == "policy":
        vocab = _spread(rng, 257, 151000)
        tokens = _spread(rng, 1, max(1, (120_000_000 if kind == "f32" else 250_000_000) // vocab))
        return {"op": op, "grad": rng.random() < 0.7, "tokens": min(tokens, 16384), "vocab": vocab, "type": kind,
                "masked": rng.choice([0.0, 0.2, 0.5])}
    inner, outer = _spread(rng, 129, 6144), _spread(rng, 129, 12288)
    return {"op": op, "backward": rng.random() < 0.5, "tokens": _spread(rng, 1, 8192), "inner": inner, "outer": outer,
            "type": rng.choice(["bf16", "f16"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _rows(g, rows, cols, pad, dtype, scale=1.0):
    """Rows of a buffer that is `pad` elements wider."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda").mul_(scale).to(dtype)
    return x[:, :cols] if pad else x


def _hidden(g, rows, cols, pad, dtype):
    """Hidden states: a few channels much larger than the rest, as trained decoders have them."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x[:, torch.randperm(cols, generator=g, device="cuda")[:max(1, cols // 256)]] *= 12.0
    x = x.to(dtype)
    return x[:, :cols] if pad else x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case), "seed": 0x9E3779B97F4A7C15 ^ (seed * 0x2545F4914F6CDD1D & (1 << 64) - 1), "offset": seed & 0xFFFF}
    op, dtype = case["op"], TYPES[case["type"]]
    if op in ("norm", "dropout"):
        rows, cols, pad = case["rows"], case["cols"], case["pad"]
        if op == "dropout":
            s["x"] = _rows(g, rows, cols, pad, dtype, 1e-3 if case["backward"] else 1.0)
            s["residual"] = _hidden(g, rows, cols, 0, dtype) if case["residual"] and not case["backward"] else None
            return s
        s["weight"] = 1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")
        s["bias"] = 0.1 * torch.randn(cols, generator=g, device="cuda")
        if case["backward"]:
            s["h"] = _hidden(g, rows, cols, pad, dtype)
            h = s["h"].float()
            s["mean"] = h.mean(1)
            s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(1) + EPS)
            s["dy"] = _rows(g, rows, cols, 0, dtype, 1e-3)
            s["dh"] = _rows(g, rows, cols, 0, dtype, 1e-3) if case["residual"] else None
        else:
            s["x"] = _rows(g, rows, cols, pad, dtype)
            s["residual"] = _hidden(g, rows, cols, 0, dtype) if case["residual"] else None
        return s
    if op == "policy":
        tokens, vocab = case["tokens"], case["vocab"]
        logits = torch.randn(tokens, vocab, generator=g, device="cuda").mul_(2.0)
        targets = torch.randint(vocab, (tokens,), generator=g, device="cuda")
        # sampled tokens are likely ones
        logits.scatter_add_(1, targets[:, None], 4.0 + 4.0 * torch.rand(tokens, 1, generator=g, device="cuda"))
        s["logits"] = logits.to(dtype)
        logp = torch.cat([torch.log_softmax(part.float(), 1).gather(1, at[:, None])[:, 0]
                          for part, at in zip(s["logits"].split(1024), targets.split(1024))])
        kept = torch.rand(tokens, generator=g, device="cuda") >= case["masked"]
        s["old"] = torch.where(kept, logp + 0.15 * torch.randn(tokens, generator=g, device="cuda"), 0.0)
        s["ref"] = torch.where(kept, logp + 0.3 * torch.randn(tokens, generator=g, device="cuda"), 0.0)
        s["advantages"] = 0.25 + torch.randn(tokens, generator=g, device="cuda")
        s["weights"] = kept.float() / kept.sum().clamp(min=1)
        s["targets"] = torch.where(kept, targets, -100)
        return s
    tokens, inner, outer = case["tokens"], case["inner"], case["outer"]
    s["x"] = _hidden(g, tokens, inner, 0, dtype)
    w = torch.randn(outer, inner, generator=g, device="cuda").mul_(0.02)
    q, e = _quantize(w, 128)
    s["w"], s["w_scale"] = _stored(q), (e + 127).to(torch.uint8).t().contiguous()
    if case["backward"]:
        spread = torch.exp(torch.randn(tokens, 1, generator=g, device="cuda"))
        s["dy"] = (torch.randn(tokens, outer, generator=g, device="cuda") * (1e-4 * spread)).to(dtype)
        s["wt"], s["wt_scale"] = _stored(q.t()), (e + 127).to(torch.uint8).contiguous()
    return s


def _stored(q):
    """An 8-bit matrix as a program keeps it: rows of a multiple of 16 bytes."""
    rows, cols = q.shape
    full = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device=q.device)
    full[:, :cols] = q.contiguous().view(torch.uint8)
    return full.view(torch.float8_e4m3fn)[:, :cols]


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

LOW = 0xFFFFFFFF


def _kept(shape, p, seed, offset):
    """The dropout's mask: element i of the row-major order is kept where word i mod 4 of Philox4x32-10 at the counter
    (i div 4, offset) under the key `seed` is at least p 2^32 (Salmon, Moraes, Dror and Shaw, SC 2011)."""
    n = math.prod(shape)
    j = torch.arange(-(-n // 4), dtype=torch.int64, device="cuda")
    c = [j & LOW, j >> 32, torch.full_like(j, offset & LOW), torch.full_like(j, offset >> 32 & LOW)]
    k0, k1 = seed & LOW, seed >> 32 & LOW
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32 & LOW) ^ c[1] ^ k0, b & LOW, (a >> 32 & LOW) ^ c[3] ^ k1, a & LOW]
        k0, k1 = k0 + 0x9E3779B9 & LOW, k1 + 0xBB67AE85 & LOW
    return (torch.stack(c, 1).reshape(-1)[:n] >= round(p * 2 ** 32)).reshape(shape)


def _dropped(x, p, seed, offset):
    return torch.where(_kept(x.shape, p, seed, offset), x * (1.0 / (1.0 - p)), 0.0) if p else x


def _norm(x, weight, bias, residual, p, seed, offset):
    h = _dropped(x.float(), p, seed, offset)
    h = (h if residual is None else h + residual.float()).to(x.dtype)
    f = h.float()
    mean = f.mean(1)
    centred = f - mean[:, None]
    rstd = 1.0 / torch.sqrt(centred.square().mean(1) + EPS)
    y = (centred * rstd[:, None] * weight + bias).to(x.dtype)
    return y, h, mean, rstd


def _norm_grad(dy, h, mean, rstd, weight, dh, p, seed, offset):
    dy, hat = dy.float(), (h.float() - mean[:, None]) * rstd[:, None]
    wdy = dy * weight
    total = rstd[:, None] * (wdy - wdy.mean(1, keepdim=True) - hat * (wdy * hat).mean(1, keepdim=True))
    total = total if dh is None else total + dh.float()
    dx = _dropped(total, p, seed, offset).to(h.dtype)
    return dx, total.to(h.dtype), (dy * hat).sum(0), dy.sum(0)


def _policy(logits, targets, old, ref, advantages, weights, grad):
    kept = weights != 0
    f = logits.float()
    at = torch.where(kept, targets, 0)[:, None]
    top = f.max(1, keepdim=True).values
    e = torch.exp(f - top)
    total = e.sum(1, keepdim=True)
    logp = torch.where(kept, (f.gather(1, at) - top - torch.log(total))[:, 0], 0.0)
    if not grad:
        return {"logp": logp}
    ratio = torch.exp(logp - old)
    clipped = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    kl = torch.exp(ref - logp) - (ref - logp) - 1
    loss = torch.where(kept, weights * (KL_COEF * kl - torch.minimum(ratio * advantages, clipped * advantages)), 0.0).sum()
    through = ratio * advantages <= clipped * advantages
    slope = torch.where(kept, weights * (KL_COEF * (1 - torch.exp(ref - logp)) - torch.where(through, ratio * advantages, 0.0)), 0.0)
    d = e / total * -slope[:, None]
    d.scatter_add_(1, at, slope[:, None])
    return {"loss": loss, "logp": logp, "dlogits": torch.where(kept[:, None], d, 0.0).to(logits.dtype)}


def _quantize(x, block_rows):
    """x in e4m3 and the exponents of its blocks' scales (block_rows by 128): the least e with all of the block within 448 2^e."""
    rows, cols = x.shape
    f = torch.nn.functional.pad(x.float(), (0, -cols % 128, 0, -rows % block_rows))
    f = f.reshape(f.shape[0] // block_rows, block_rows, f.shape[1] // 128, 128)
    m, k = torch.frexp(f.abs().amax((1, 3)))
    e = torch.where(m > 0, k - 9 + (m > 0.875).to(torch.int32), -127).clamp(min=-127)
    back = (127 - e << 23).view(torch.float32)[:, None, :, None]
    q = (f * back).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(q.shape[0] * block_rows, -1)[:rows, :cols].view(torch.float8_e4m3fn), e


def _values(q, scale, block_rows):
    """What an 8-bit matrix stands for; scale: a byte for each block, its exponent plus 127, column blocks first."""
    rows, cols = q.shape
    v = torch.where(scale > 0, scale.to(torch.int32) << 23, 1 << 22).view(torch.float32).t()
    return q.float() * v.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def _rounded(x, block_rows=1):
    q, e = _quantize(x, block_rows)
    return _values(q, (e + 127).to(torch.uint8).t(), block_rows)


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        from matrix_optimizer_step_rot_gb300 import operators as ops
    if op == "norm" and not c["backward"]:
        if own:
            y, h, mean, rstd = ops.layer_norm(s["x"], s["weight"], s["bias"], EPS, residual=s["residual"], p=c["p"],
                                              seed=s["seed"], offset=s["offset"])
        else:
            y, h, mean, rstd = _norm(s["x"], s["weight"], s["bias"], s["residual"], c["p"], s["seed"], s["offset"])
        return {"y": y, "h": h, "mean": mean, "rstd": rstd}
    if op == "norm":
        if own:
            dx, total, dw, db = ops.layer_norm_backward(s["dy"], s["h"], s["mean"], s["rstd"], s["weight"], dh=s["dh"],
                                                        p=c["p"], seed=s["seed"], offset=s["offset"])
        else:
            dx, total, dw, db = _norm_grad(s["dy"], s["h"], s["mean"], s["rstd"], s["weight"], s["dh"], c["p"],
                                           s["seed"], s["offset"])
        return {"dx": dx, "dh": total, "dweight": dw, "dbias": db}
    if op == "dropout":
        if own:
            if c["backward"]:
                return {"y": ops.dropout_backward(s["x"], c["p"], s["seed"], s["offset"])}
            return {"y": ops.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"])}
        y = _dropped(s["x"].float(), c["p"], s["seed"], s["offset"])
        return {"y": (y if s["residual"] is None else y + s["residual"].float()).to(s["x"].dtype)}
    if op == "policy":
        if not own:
            return _policy(s["logits"], s["targets"], s["old"], s["ref"], s["advantages"], s["weights"], c["grad"])
        if not c["grad"]:
            return {"logp": ops.token_logprobs(s["logits"], s["targets"], weights=s["weights"])}
        loss, logp, d = ops.policy_loss(s["logits"], s["targets"], s["old"], s["advantages"], s["weights"], ref_logp=s["ref"],
                                        clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL_COEF)
        return {"loss": loss, "logp": logp, "dlogits": d}
    if own:
        if not c["backward"]:
            return {"y": ops.fp8_linear(s["x"], ops.Fp8Matrix(s["w"], s["w_scale"], 128))}
        dx, dw = ops.fp8_linear_backward(s["dy"], s["x"], ops.Fp8Matrix(s["wt"], s["wt_scale"], 128))
        return {"dx": dx, "dw": dw}
    if not c["backward"]:
        return {"y": (_rounded(s["x"]) @ _values(s["w"], s["w_scale"], 128).t()).to(s["x"].dtype)}
    dx = (_rounded(s["dy"]) @ _values(s["wt"], s["wt_scale"], 128).t()).to(s["dy"].dtype)
    return {"dx": dx, "dw": _rounded(s["dy"].t()) @ _rounded(s["x"].t()).t()}


def work(case):
    es, op = BYTES[case["type"]], case["op"]
    if op in ("norm", "dropout"):
        rows, cols, p, residual = case["rows"], case["cols"], case["p"], case["residual"]
        n = rows * cols
        if op == "dropout":
            return {"bytes": n * es * (3 if residual and not case["backward"] else 2), "flops": 2 * n}
        if case["backward"]:  # dy, h and the stream's gradient in, one gradient or (with dropout) two out
            return {"bytes": n * es * (2 + residual + 1 + (p > 0)) + 12 * cols + 8 * rows, "flops": 14 * n}
        # x and the residual in, y out, and the stream where it is not x itself
        return {"bytes": n * es * (2 + residual + (residual or p > 0)) + 8 * cols + 8 * rows, "flops": 9 * n}
    if op == "policy":
        n, kept = case["tokens"] * case["vocab"], 1.0 - case["masked"]
        return {"bytes": int(n * es * (kept + case["grad"])) + 28 * case["tokens"], "flops": int(n * kept * (9 if case["grad"] else 5))}
    t, i, o = case["tokens"], case["inner"], case["outer"]
    if case["backward"]:
        return {"bytes": t * o * es + 2 * t * i * es + i * o * 5, "flops": 4 * t * i * o}
    return {"bytes": t * (i + o) * es + i * o, "flops": 2 * t * i * o}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_kept(count, p, seed, offset):
    """The mask of the first `count` elements, by whole numbers in 16-bit halves."""
    def product(x, m):
        x0, x1, m0, m1 = x & 0xFFFF, x >> 16, m & 0xFFFF, m >> 16
        mid = x1 * m0 + (x0 * m0 >> 16)
        low = x0 * m1 + (mid & 0xFFFF)
        return x1 * m1 + (mid >> 16) + (low >> 16), (low & 0xFFFF) << 16 | x0 * m0 & 0xFFFF

    i = torch.arange((count + 3) // 4, device="cuda")
    w0, w1 = i % 2 ** 32, i // 2 ** 32
    w2, w3 = torch.zeros_like(i) + offset % 2 ** 32, torch.zeros_like(i) + offset // 2 ** 32
    for r in range(10):
        key0, key1 = (seed + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        hi0, lo0 = product(w0, 0xD2511F53)
        hi2, lo2 = product(w2, 0xCD9E8D57)
        w0, w1, w2, w3 = hi2 ^ w1 ^ key0, lo2, hi0 ^ w3 ^ key1, lo0
    words = torch.empty(i.numel(), 4, dtype=torch.int64, device="cuda")
    for k, w in enumerate((w0, w1, w2, w3)):
        words[:, k] = w
    return words.flatten()[:count].double() >= float(round(p * 2.0 ** 32))


def _exact_dropped(x, c, s):
    if not c["p"]:
        return x
    kept = _exact_kept(x.numel(), c["p"], s["seed"], s["offset"]).view(x.shape)
    return torch.where(kept, x / (1.0 - c["p"]), torch.zeros_like(x))


def _two_to(e):
    """2^e of whole numbers e in 64 bits, to the last bit."""
    return (e.to(torch.int64) + 1023 << 52).view(torch.float64)


def _exact_rounded(x, block_rows=1):
    """Each block of block_rows by 128 on the grid of four significant bits, exponents from -6 up, under its scale."""
    x = x.double()
    out = torch.empty_like(x)
    for at in range(0, x.shape[1], 128):
        part = x[:, at:at + 128]
        top = part.abs().amax(1)
        if block_rows > 1:
            top = torch.cat([b.max().expand(b.shape[0]) for b in top.split(block_rows)])
        e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -300)))
        for _ in range(2):  # the logarithm's rounding may be one off
            e = torch.where(top > 448.0 * _two_to(e), e + 1, e)
            e = torch.where(top <= 448.0 * _two_to(e - 1), e - 1, e)
        scale = _two_to(e.clamp(min=-127))[:, None]
        v = part / scale
        size = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(min=-6)
        size = torch.where(v.abs() < _two_to(size), size - 1, size).clamp(min=-6)
        step = _two_to(size - 3)
        out[:, at:at + 128] = torch.round(v / step) * step * scale
    return out


def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "dropout":
        y = _exact_dropped(s["x"].double(), c, s)
        return {"y": y if s["residual"] is None else s["residual"].double() + y}
    if op == "norm" and not c["backward"]:
        h = _exact_dropped(s["x"].double(), c, s)
        h = h if s["residual"] is None else s["residual"].double() + h
        f = h.to(s["x"].dtype).double()  # the norm reads the stream as it is kept
        var, mean = torch.var_mean(f, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = (f - mean.unsqueeze(1)) * rstd.unsqueeze(1) * s["weight"].double() + s["bias"].double()
        return {"y": y, "h": h, "mean": mean, "rstd": rstd}
    if op == "norm":
        h, dy, n = s["h"].double(), s["dy"].double(), c["cols"]
        rstd = s["rstd"].double().unsqueeze(1)
        hat = (h - s["mean"].double().unsqueeze(1)) * rstd
        wdy = dy * s["weight"].double()
        total = rstd / n * (n * wdy - wdy.sum(1, keepdim=True) - hat * (wdy * hat).sum(1, keepdim=True))
        if s["dh"] is not None:
            total = total + s["dh"].double()
        return {"dx": _exact_dropped(total, c, s), "dh": total, "dweight": torch.einsum("rc,rc->c", dy, hat), "dbias": dy.sum(0)}
    if op == "policy":
        logp, d, loss = [], [], 0.0
        for at in range(0, c["tokens"], 512):
            f = s["logits"][at:at + 512].double()
            w = s["weights"][at:at + 512].double()
            kept = w != 0
            t = s["targets"][at:at + 512].clamp(min=0)
            full = torch.log_softmax(f, 1)
            lp = full[torch.arange(f.shape[0], device="cuda"), t] * kept
            logp.append(lp)
            if not c["grad"]:
                continue
            old, ref, adv = (s[k][at:at + 512].double() for k in ("old", "ref", "advantages"))
            ratio = (lp - old).exp()
            bounded = torch.where(adv >= 0, ratio.clamp(max=1 + CLIP_HIGH), ratio.clamp(min=1 - CLIP_LOW))
            r = ref - lp
            loss = loss + (w * (KL_COEF * (torch.expm1(r) - r) - bounded * adv)).sum()
            slope = w * (-KL_COEF * torch.expm1(r) - ratio * adv * (bounded == ratio))
            part = -slope[:, None] * full.exp()
            part[torch.arange(f.shape[0], device="cuda"), t] += slope
            d.append((part * kept[:, None]).to(torch.float32 if c["type"] != "f32" else torch.float64))
        if not c["grad"]:
            return {"logp": torch.cat(logp)}
        return {"loss": loss, "logp": torch.cat(logp), "dlogits": torch.cat(d)}
    if not c["backward"]:
        w = s["w"].double() * _two_to(s["w_scale"].int() - 127).t().repeat_interleave(128, 0)[:c["outer"]] \
            .repeat_interleave(128, 1)[:, :c["inner"]]
        return {"y": _exact_rounded(s["x"]) @ w.t()}
    w = s["wt"].double() * _two_to(s["wt_scale"].int() - 127).t().repeat_interleave(128, 0)[:c["inner"]] \
        .repeat_interleave(128, 1)[:, :c["outer"]]
    dx = _exact_rounded(s["dy"]) @ w.t()
    return {"dx": dx, "dw": _exact_rounded(s["dy"].t().contiguous()) @ _exact_rounded(s["x"].t().contiguous()).t()}
