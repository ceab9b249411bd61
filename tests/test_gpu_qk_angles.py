"""The rotation's angles at far positions, against exact arithmetic: negative frequencies, and ones so small that
their 64-bit fraction of a turn has few digits.

Bound in turns (as documented): |p f| 2^-53 + |p| 2^-65 + 2^-25.  x = (1, 0) for every pair, so that the outputs are the
cosine and the sine; they add 4 u (u = 2^-24: sine and cosine 2 u, the products with 1 and 0 and the last rounding)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
FREQ = [-1e-6, 2.3e-7, -2.3e-7, -0.25, 1e-4, -1e-12, 3e-9, -7.0, 1e-18, -1e-18, 0.0, 1.0, -6.283185307179586,
        2.46e-6, -5e-324, 100.0]
POS = [0, 1, -1, 4999, 1 << 24, 1 << 34, -(1 << 34) - 3, (1 << 40) + 12345, -(1 << 40), (1 << 45) + 1, -(1 << 45) - 7]


def exact(p, f):
    """cos and sin of p f."""
    turns = Fraction(p) * Fraction(f) / (2 * PI)
    turns -= turns.numerator // turns.denominator
    phi = 2 * np.pi * float(turns - 1 if turns > Fraction(1, 2) else turns)
    return np.cos(phi), np.sin(phi)


@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_far_positions(gpu_lib, layout):
    D, T = 2 * len(FREQ), len(POS)
    p = gpu_lib.ShardedAttentionProj(T, 64, [D], [D], "fp32")
    p.set_qk_norm_rope(D, layout=layout, norm=False, inv_freq=FREQ)
    a = slice(0, D // 2) if layout == "halves" else slice(0, D, 2)
    b = slice(D // 2, D) if layout == "halves" else slice(1, D, 2)
    x = torch.zeros(T, 3 * D, device="cuda")
    x[:, :D][:, a] = 1
    pos = torch.tensor(POS, device="cuda")
    y = p.qk_norm_rope_forward([x], pos)[0].double().cpu().numpy()[:, :D]
    back = p.qk_norm_rope_backward([x], [x[:, :2 * D].contiguous()], pos, dV_i=[x[:, :D].contiguous()])[0][0]
    back = back.double().cpu().numpy()[:, :D]
    for i, at in enumerate(POS):
        for j, f in enumerate(FREQ):
            c, s = exact(at, f)
            turns = abs(at * f) * 2.0 ** -53 + abs(at) * 2.0 ** -65 + 2.0 ** -25
            bound = 2 * np.pi * turns + 4 * 2.0 ** -24
            got = [v[i][side][j] for v in (y, back) for side in (a, b)]
            assert np.abs(np.array(got) - [c, s, c, -s]).max() <= bound, (at, f, got, c, s, bound)
