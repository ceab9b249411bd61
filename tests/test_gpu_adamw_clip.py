"""Clipping where grad_scale takes the gradients' norm to the end of the fp32 range and past it."""
import pytest
import torch

from test_gpu_adamw import Copy, check_step, make

pytestmark = pytest.mark.gpu

SIZES = [7, 300, 5000]


def optimizer(tp, bits, max_norm):
    p, grads = make(SIZES, "fp32", "fp32")
    g = [x * 1e4 for x in grads(0)]  # a norm of some hundreds
    return tp.ShardedAdamW(p, lr=1e-3, bits=bits, max_norm=max_norm), g


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [1e30, 1e36, 1e38, 3e38])
def test_a_clipped_norm_may_pass_the_range(gpu_lib, bits, scale):
    opt, g = optimizer(gpu_lib, bits, 1.0)
    for _ in range(2):
        old = Copy(opt)
        check_step(opt, old, g, opt.step(g, grad_scale=scale), [0.0] * len(SIZES), scale)


@pytest.mark.parametrize("bits", [32, 8])
def test_without_clipping_the_step_is_skipped(gpu_lib, bits):
    opt, g = optimizer(gpu_lib, bits, float("inf"))
    before = [x.clone() for x in opt.params + opt.m + opt.v]
    norm = opt.step(g, grad_scale=3e38)
    assert torch.isfinite(norm)
    assert all(torch.equal(a, b) for a, b in zip(before, opt.params + opt.m + opt.v))
    old = Copy(opt)
    check_step(opt, old, g, opt.step(g, grad_scale=1e-3), [0.0] * len(SIZES), 1e-3)
