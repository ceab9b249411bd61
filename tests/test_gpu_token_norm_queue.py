"""The tokens' norm with many tokens a team, so that every stage of a thread's queue is refilled and both halves of the
team's sums are used again, against the definition in 64 bits; bounds as in the tests of single tokens."""
import pytest
import torch

from test_gpu_token_norm import EPS, U, check_backward, check_forward, half, make, within

pytestmark = pytest.mark.gpu

# A CTA of 16 warps an SM: teams of 1, 2, 4, 8 and 16 warps, 160 x 16 / W of them at most; each width's team gets more
# tokens than its queue has stages (forward 6 to 4 for the narrowest, then fewer; backward 2 or 1), with whole and three quarter loads of a thread, and widths that fill no round of threads.
SHAPES = [(20_000, 40), (30_000, 256), (15_000, 504), (10_000, 768), (10_000, 1000), (5_000, 1544), (4_000, 2048),
          (2_600, 2568), (2_500, 4096), (1_400, 5000), (1_000, 8192), (700, 10_000), (500, 16_384)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("T,d", SHAPES)
def test_many_tokens_a_team(gpu_lib, T, d, add, kind, dtype):
    a = make(T, d, dtype, seed=T + d)
    norm = gpu_lib.TokenNorm(T, d, kind, dtype, eps=EPS)
    bias = a["b"] if kind == "layer" else None
    y, stats, s = norm.forward(a["x"], a["g"], bias, residual=a["r"] if add else None)
    if add:
        exact = a["x"].double() + a["r"].double()
        within(s, exact, (half(dtype) * 1.001 + U) * exact.abs())
    check_forward(y, stats, s, a["g"], bias, kind, dtype)
    ds = a["ds"] if add else None
    check_backward(norm.backward(s, stats, a["dy"], a["g"], dsum=ds, bias_grad=kind == "layer"), s, stats, a["dy"], ds,
                   a["g"], kind, dtype)


@pytest.mark.parametrize("T,d,kind", [(8192, 4096, "rms"), (8192, 16_384, "rms"), (8192, 768, "layer"), (65_536, 256, "layer")])
def test_batches(gpu_lib, T, d, kind):
    test_many_tokens_a_team(gpu_lib, T, d, True, kind, "bf16")
