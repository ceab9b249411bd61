"""Plain 64-bit torch forms of the tokens' norm, for the tests."""
import torch


def norm_forward(s, gain, bias, kind, eps):
    """y, mu [T], r [T] of s [T, d]; gain, bias: [d] or None."""
    s = s.double()
    mu = s.mean(1) if kind == "layer" else torch.zeros_like(s[:, 0])
    c = s - mu[:, None]
    r = 1 / ((c * c).mean(1) + eps).sqrt()
    y = c * r[:, None]
    if gain is not None:
        y = y * gain.double()
    if bias is not None:
        y = y + bias.double()
    return y, mu, r


def norm_backward(s, mu, r, dy, dsum, gain, kind):
    """dx, dgain, dbias from the statistics; dsum, gain: or None."""
    s, dy = s.double(), dy.double()
    n = (s - mu.double()[:, None]) * r.double()[:, None]
    w = dy if gain is None else dy * gain.double()
    dx = w - n * (w * n).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - w.mean(1, keepdim=True)
    dx = dx * r.double()[:, None]
    if dsum is not None:
        dx = dx + dsum.double()
    return dx, (dy * n).sum(0), dy.sum(0)


# ---------------------------------------------------------------- AdamW

GROUP = 256
MASK = (1 << 32) - 1


def adamw(p, g, m, v, t, lr, b1, b2, eps, decay, f=1.0):
    """p, m, v after step t, in 64 bits."""
    p, g, m, v = p.double(), g.double() * f, m.double(), v.double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    return p - lr * decay * p - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps), m, v


def mix(x):
    x = ((x ^ (x >> 16)) * 0x7feb352d) & MASK
    x = ((x ^ (x >> 15)) * 0x846ca68b) & MASK
    return x ^ (x >> 16)


def pow2(e):
    """2^e of integers in the normal range, from the bits: ldexp and exp2 on the device are a last place off."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def randoms(seed, step, group0, groups, device="cpu"):
    """The 16 random bits of every element of groups group0, group0 + 1, ...: [groups, 256]."""
    key = mix(mix(mix(mix(seed & MASK) ^ (seed >> 32)) ^ (step & MASK)) ^ (step >> 32))
    q = torch.arange(group0, group0 + groups, device=device)[:, None]
    a = mix(mix(key ^ (q & MASK)) ^ (q >> 32))
    l = torch.arange(GROUP, device=device)[None]
    h = mix((a + (l // 2) * 0x9e3779b9) & MASK)
    return torch.where(l % 2 == 0, h & 0xffff, h >> 16)


def exponent(most):
    """e of groups whose largest magnitudes these are (positive, 64 bits)."""
    man, ex = torch.frexp(most)  # most = man 2^ex, man in [0.5, 1)
    return (ex - 1 + (man * 2 > 1.875).int()).clamp_min(-90)


def rounded(x, e, r, second):
    """What x [groups, 256] is kept as, with its groups' e [groups] and the elements' random bits."""
    S = 31 if second else 15
    a = x.abs()
    least = 1.125 * pow2(e - S)[:, None].expand_as(a)
    man, ex = torch.frexp(a)
    eighths = man * 16
    low = eighths.floor()
    up = (eighths - low >= 1 - r / 65536).double()
    kept = (low + up) / 8 * pow2(ex - 1)
    small = (a > 0) if second else a * 65536 > least * r
    kept = torch.where(a < least, torch.where(small, least, 0.0), kept)
    return torch.where(x < 0, -kept, kept)


def values(buf, n, second):
    """(values [n] in 64 bits, scale bytes) of a stored moment."""
    S = 31 if second else 15
    groups = -(-n // GROUP)
    c, b = buf[:groups * GROUP].view(groups, GROUP).long(), buf[groups * GROUP:]
    mag = c if second else c & 127
    e = b.long()[:, None] - 91
    v = (1 + (mag & 7) / 8).double() * pow2((mag >> 3) + e - S)
    v = torch.where(mag == 0, 0.0, v)
    if not second:
        v = torch.where(c > 127, -v, v)
    v = torch.where(b[:, None] == 255, float("nan"), v)
    return v.view(-1)[:n], b
