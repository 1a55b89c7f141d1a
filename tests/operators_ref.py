"""Plain 64-bit restatements of the operators (include/rot_ops.h), for their tests."""

import numpy as np
import torch


def philox(counter, offset, seed):
    """Philox4x32-10 on arrays of 64-bit counters: [n, 4] uint32 words."""
    counter = np.asarray(counter, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    c = [counter & low, counter >> sh, np.full_like(counter, offset & 0xFFFFFFFF),
         np.full_like(counter, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k0), b & low, (a >> sh) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).astype(np.uint32)


def kept(first, count, p, seed, offset):
    """The mask of elements first .. first + count - 1 (first a multiple of 4)."""
    assert first % 4 == 0
    j = np.arange(first // 4, (first + count + 3) // 4, dtype=np.uint64)
    words = philox(j, offset, seed).reshape(-1)[:count]
    return words.astype(np.uint64) >= np.uint64(np.rint(p * 2.0 ** 32))


def dropped(x, p, seed, offset):
    """float64 of x (any shape) with dropout, on x's device."""
    x = x.double()
    if p == 0:
        return x
    k = torch.from_numpy(kept(0, x.numel(), p, seed, offset)).to(x.device).view(x.shape)
    scale = float(np.float32(1.0 / (1.0 - p))) if p < 1 else 0.0
    return torch.where(k, x * scale, torch.zeros_like(x))


def norm(h, weight, bias, eps):
    """(y, mean, rstd, hat) of rows h."""
    h = h.double()
    mean = h.mean(1)
    var = (h - mean[:, None]).square().mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    hat = (h - mean[:, None]) * rstd[:, None]
    y = hat * weight.double()
    return (y if bias is None else y + bias.double()), mean, rstd, hat


def norm_grad(dy, hat, rstd, weight, dh):
    """(gradient of h, dweight, dbias)."""
    dy = dy.double()
    wdy = dy * weight.double()
    g = rstd[:, None] * (wdy - wdy.mean(1, keepdim=True) - hat * (wdy * hat).mean(1, keepdim=True))
    if dh is not None:
        g = g + dh.double()
    return g, (dy * hat).sum(0), dy.sum(0)


def policy(logits, targets, old, ref, adv, w, lo, hi, kl):
    """(loss, logp, terms, gradient) by the formulas, over the unmasked tokens."""
    z = logits.double()
    logp, terms, grad = torch.zeros(len(z)).double(), torch.zeros(len(z)).double(), torch.zeros_like(z)
    logp, terms = logp.to(z.device), terms.to(z.device)
    on = (w != 0).nonzero()[:, 0]
    z, t = z[on], targets[on]
    full = z - torch.logsumexp(z, 1, keepdim=True)
    lp = full.gather(1, t[:, None])[:, 0]
    logp[on] = lp
    if old is None:
        return None, logp, None, None
    old, adv, wd = old[on].double(), adv[on].double(), w[on].double()
    ratio = torch.exp(lp - old)
    plain, clipped = ratio * adv, ratio.clamp(1 - lo, 1 + hi) * adv
    v = -torch.minimum(plain, clipped)
    s = -torch.where(plain <= clipped, plain, torch.zeros_like(plain))
    if ref is not None:
        r = ref[on].double() - lp
        v = v + kl * (torch.expm1(r) - r)
        s = s - kl * torch.expm1(r)
    terms[on] = wd * v
    g = -(wd * s)[:, None] * torch.exp(full)
    g.scatter_add_(1, t[:, None], (wd * s)[:, None])
    grad[on] = g
    return terms.sum(), logp, terms, grad


# ---- 8-bit matrices ----

FORMATS = {torch.float8_e4m3fn: (448.0, 3, -6), torch.float8_e5m2: (57344.0, 2, -14)}


def quantize(x, block_rows, dtype):
    """(values in 8-bit units as float64, scale bytes [ceil(C/128), ceil(R/block_rows)]) of a numpy
    array, block by block, by the definition."""
    top, bits, least = FORMATS[dtype]
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    q = np.zeros_like(x)
    scale = np.zeros((-(-C // 128), -(-R // block_rows)), dtype=np.uint8)
    for j in range(scale.shape[0]):
        for i in range(scale.shape[1]):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128))
            b = x[at]
            fine = np.isfinite(b)
            big = np.abs(b[fine]).max() if fine.any() else 0.0
            e = -127
            while big > top * 2.0 ** e:
                e += 1
            scale[j, i] = e + 127
            v = np.where(fine, b, 0.0) * 2.0 ** -e
            _, ex = np.frexp(v)  # v = m 2^ex, m in [1/2, 1)
            step = 2.0 ** (np.maximum(ex - 1, least) - bits)
            q[at] = np.where(fine, np.round(v / step) * step, np.nan)
    return q, scale


def scale_of(byte):
    """2^(byte - 127) as float64; 255 is NaN."""
    e = byte.to(torch.int64) - 127
    v = (e + 1023 << 52).view(torch.float64)
    return torch.where(byte == 255, torch.full_like(v, float("nan")), v)


def values(m):
    """float64 matrix that an Fp8Matrix stands for."""
    rows, cols = m.data.shape
    s = scale_of(m.scale).t().repeat_interleave(m.block_rows, 0)[:rows]
    return m.data.to(torch.float32).double() * s.repeat_interleave(128, 1)[:, :cols]
