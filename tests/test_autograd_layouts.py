"""The autograd functions with tensors that the library cannot read as they lie: they are copied first."""
import pytest
import torch

import megatron_tensor_transformer_column_gb300 as tp

TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


def odd(x):
    """x, contiguous, one element off 16 bytes."""
    flat = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)
    flat[1:] = x.flatten()
    return flat[1:].view(x.shape)


def test_dense():
    x = torch.arange(48.0).view(6, 8)
    assert tp._dense(x) is x
    for y in (odd(x), x.t().contiguous().t(), torch.cat([x, x], 1)[:, 1:9], torch.cat([x, x], 1)[:, 8:], x[:0]):
        z = tp._dense(y)
        assert z.is_contiguous() and z.data_ptr() % 16 == 0 and torch.equal(z, y)


def leaves(gen, shapes, dtype):
    return [(0.3 * torch.randn(*s, generator=gen, device="cuda")).to(TD[dtype]) for s in shapes]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(gpu_lib, dtype, residual):
    T, d = 24, 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, r, dy = leaves(gen, [(T, d)] * 3, dtype)
    g, b = leaves(gen, [(d,)] * 2, dtype)
    norm = gpu_lib.TokenNorm(T, d, "layer", dtype)

    def run(lay, wrap):
        a = [lay(t).detach().requires_grad_() for t in ((x, r) if residual else (x,))]
        p = [t.clone().requires_grad_() for t in (g, b)]
        y = gpu_lib.TPMLPNormFunction.apply(norm, a[0], *p, *a[1:])
        return torch.autograd.grad(wrap(y), a + p)

    dense = lambda y: sum((t * dy).sum() for t in y) if residual else (y * dy).sum()
    want = run(lambda t: t, dense)
    for lay in (odd, lambda t: torch.cat([t[:, :2], t, t[:, :2]], 1)[:, 2:-2]):
        assert all(torch.equal(u, v) for u, v in zip(want, run(lay, dense)))

    def behind(y):  # the gradient arrives as columns 2 .. 65 of 68, at an odd start with rows on 16 bytes
        return sum((torch.cat([t.new_zeros(T, 2), t, t.new_zeros(T, 2)], 1) * torch.nn.functional.pad(dy, (2, 2))).sum()
                   for t in (y if residual else (y,)))

    def flat(y):  # a contiguous gradient at an odd start
        return sum((torch.cat([t.new_zeros(1), t.flatten()]) * torch.nn.functional.pad(dy.flatten(), (1, 0))).sum()
                   for t in (y if residual else (y,)))

    for wrap in (behind, flat):
        assert all(torch.equal(u, v) for u, v in zip(want, run(lambda t: t, wrap)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("name", ["TPMLPFunction", "TPMLPCheckpointFunction", "TPMLPResidualFunction"])
def test_blocks(gpu_lib, name, act, dtype):
    T, d, widths = 40, 64, [64, 32]
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, r, dy = leaves(gen, [(T, d)] * 3, dtype)
    ws = leaves(gen, [(d, w) for w in widths] + [(w, d) for w in widths] +
                ([(d, w) for w in widths] if act == "swiglu" else []), dtype)
    mlp = gpu_lib.ShardedMLP(T, d, widths, act, dtype)
    fn = getattr(gpu_lib, name)

    def run(lay, wrap):
        a = [lay(t).detach().requires_grad_() for t in ((x, r) if "Residual" in name else (x,))]
        p = [w.clone().requires_grad_() for w in ws]
        return torch.autograd.grad(wrap(fn.apply(mlp, *a, *p)), a + p)

    want = run(lambda t: t, lambda y: (y * dy).sum())
    for lay in (odd, lambda t: torch.cat([t[:, :2], t], 1)[:, 2:], lambda t: t.t().contiguous().t()):
        assert all(torch.equal(u, v) for u, v in zip(want, run(lay, lambda y: (y * dy).sum())))
    wrap = lambda y: (torch.cat([y.new_zeros(1), y.flatten()]) * torch.nn.functional.pad(dy.flatten(), (1, 0))).sum()
    assert all(torch.equal(u, v) for u, v in zip(want, run(lambda t: t, wrap)))
