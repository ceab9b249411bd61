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
