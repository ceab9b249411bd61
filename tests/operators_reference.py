"""Plain 64-bit numpy forms of the head norm with rotation and of the 8-bit checkpoints, for the tests."""
import numpy as np


# ---------------------------------------------------------------- norm and rotation of one side's heads

def pairs_of(R, layout):
    j = np.arange(R // 2)
    return (j, j + R // 2) if layout == "halves" else (2 * j, 2 * j + 1)


def rotate(x, pos, freq, layout, sign=1.0):
    """x [T, H, D] rotated by pos * freq (freq: R / 2 radians per position)."""
    ia, ib = pairs_of(2 * len(freq), layout)
    phi = sign * np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    c, s = np.cos(phi), np.sin(phi)
    y = x.copy()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def rotate_abs(x, R, layout):
    """|a| + |b| of an element's pair (its own magnitude where it is not rotated)."""
    ia, ib = pairs_of(R, layout)
    y = np.abs(x)
    both = y[..., ia] + y[..., ib]
    y[..., ia] = both
    y[..., ib] = both
    return y


def heads_forward(x, pos, freq, layout, g, eps, norm=True):
    """y of x [T, H, D], and the magnitude its rounding errors are relative to."""
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) if norm else 1.0
    u = x * r * g
    return rotate(u, pos, freq, layout), rotate_abs(u, 2 * len(freq), layout)


def heads_backward(x, dy, pos, freq, layout, g, eps, norm=True):
    """dx, dg and the magnitudes their rounding errors are relative to."""
    w = rotate(dy, pos, freq, layout, -1.0)
    wabs = rotate_abs(dy, 2 * len(freq), layout)
    if not norm:
        return w, None, wabs, None
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n = x * r
    dg = (w * n).sum((0, 1))
    s = w * g
    dx = r * (s - n * np.mean(s * n, -1, keepdims=True))
    sabs = wabs * np.abs(g)
    dx_abs = r * (32 * sabs + 80 * np.abs(n) * np.mean(sabs * np.abs(n), -1, keepdims=True))
    return dx, dg, dx_abs, (wabs * np.abs(n)).sum((0, 1))


def frequencies(R, base=10000.0):
    return base ** (-2.0 * np.arange(R // 2) / max(R, 1))


# ---------------------------------------------------------------- 8-bit checkpoints

def _e4m3_table():
    code = np.arange(127)
    ex, man = code >> 3, code & 7
    return np.where(ex > 0, (1 + man / 8.0) * 2.0 ** (ex - 7.0), man / 8.0 * 2.0 ** -6)


E4M3 = _e4m3_table()  # the finite magnitudes, codes 0 .. 126


def encode(v):
    """e4m3 codes of finite v (|v| <= 448): the nearest number of the table, the even code on a tie."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def pack(x):
    """(codes [rows, G, 16], scale bytes [rows, G]) of x [rows, cols]; codes of a bad group are 0 here."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    G = -(-cols // 16)
    g = np.zeros((rows, G * 16))
    g[:, :cols] = x
    g = g.reshape(rows, G, 16)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    m = np.abs(g).max(-1)
    e = np.full(m.shape, -117)
    for i in range(-117, 121):  # the smallest e with m <= 448 * 2^e
        e = np.where(m > 448.0 * 2.0 ** (i - 1), np.maximum(e, i), e)
    e = np.minimum(e, 120)
    v = g / 2.0 ** e[..., None].astype(np.float64)
    v = np.where((e == 120)[..., None], np.clip(v, -240, 240), v)
    return encode(v), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scale, cols):
    v = E4M3[np.minimum(codes & 127, 126)] * np.where(codes & 128, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(codes.shape[0], -1)[:, :cols]


def nbytes(rows, cols):
    return -(-rows // 32) * -(-cols // 16) * 544


def split(buf, rows, cols):
    """Storage -> (codes [rows, G, 16], scale bytes [rows, G])."""
    B, G = -(-rows // 32), -(-cols // 16)
    n = B * G * 512
    c = buf[:n].reshape(B, G, 32, 16).transpose(0, 2, 1, 3).reshape(B * 32, G, 16)
    s = buf[n:].reshape(B, G, 32).transpose(0, 2, 1).reshape(B * 32, G)
    return c[:rows], s[:rows]


def pad_bytes(buf, rows, cols):
    """The stored bytes that stand for rows past the last."""
    B, G = -(-rows // 32), -(-cols // 16)
    n = B * G * 512
    c = buf[:n].reshape(B, G, 32, 16).transpose(0, 2, 1, 3).reshape(B * 32, -1)
    s = buf[n:].reshape(B, G, 32).transpose(0, 2, 1).reshape(B * 32, G)
    return np.concatenate([c[rows:].ravel(), s[rows:].ravel()])
