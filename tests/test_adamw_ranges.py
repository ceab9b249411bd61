"""AdamW at the ends of the fp32 range: numbers that it does not hold are refused, second moments below 2^-126 count.

Bounds as in the tests of whole steps (u = 2^-24: m 4 u b1 |m| + 12 u (1 - b1) |f g|, v 24 u, the update 26 u and 1 u for
a root that may be flushed), and 2^-148 for m and v each, whose at most three roundings below 2^-126 are 2^-150 each."""
import math

import pytest
import torch

import megatron_tensor_transformer_column_gb300 as tp
import step_reference as ref
from test_step_operators_cpu import CUDA, FAKE, INVALID, status_of, step_call

U = 2.0 ** -24
TINY = 2.0 ** -126
FLUSH = 2.0 ** -38 / math.sqrt(1 - 0.999)  # an eps from here on may flush v


@pytest.fixture(scope="module")
def lib():
    from megatron_tensor_transformer_column_gb300 import _build
    _build.build()
    return tp.load()


def test_numbers_that_fp32_does_not_hold_are_refused(lib):
    call = lambda norm=8 * FAKE, weight_decay=None, **hyper: step_call(hyper=hyper, norm=norm, weight_decay=weight_decay)
    for h in (dict(eps=1e-39), dict(eps=1e-50), dict(eps=1e39), dict(eps=TINY * (1 - 1e-9)), dict(lr=1e39), dict(lr=-1e39),
              dict(grad_scale=1e39), dict(max_norm=1e-39), dict(max_norm=1e-50), dict(lr=1e38, beta1=0.999),
              dict(weight_decay=[0.1, 1e39]), dict(weight_decay=[0.1, -1e39]), dict(weight_decay=[1e20, 0.0], lr=1e20)):
        assert status_of(lambda: call(**h)) == INVALID
    if not torch.cuda.is_available():
        for h in (dict(eps=TINY), dict(lr=0.0), dict(lr=-1e-3), dict(grad_scale=1e38), dict(grad_scale=0.0),
                  dict(max_norm=float("inf")), dict(max_norm=TINY), dict(max_norm=1e50), dict(lr=1e39, lr_device=9 * FAKE),
                  dict(weight_decay=[1e20, 0.0], lr=1e20, lr_device=9 * FAKE), dict(weight_decay=[0.0, 1e-50]),
                  dict(beta1=0.0, beta2=0.0)):
            assert status_of(lambda: call(**h)) == CUDA  # the arguments are good


def check(opt, g, steps):
    b1, b2 = opt.betas
    for _ in range(steps):
        if opt.bits == 32:
            m0, v0 = opt.m[0].double(), opt.v[0].double()
        else:
            m0, v0 = (ref.values(b[0], g.numel(), second)[0] for b, second in ((opt.m, False), (opt.v, True)))
        weight = (opt.master or opt.params)[0]
        weight.zero_()
        opt.step([g])
        t, x = opt.steps, g.double()
        m, v = b1 * m0 + (1 - b1) * x, b2 * v0 + (1 - b2) * x * x
        dm = 4 * U * b1 * m0.abs() + 12 * U * (1 - b1) * x.abs() + 2.0 ** -148
        dv = 24 * U * v + 2.0 ** -148
        den = [((v + s * dv).clamp_min(0) / (1 - b2 ** t)).sqrt() + opt.eps for s in (1, -1)]
        least = (m.abs() - dm).clamp_min(0) / den[0] * (1 - 27 * U)
        most = (m.abs() + dm) / den[1] * (1 + 27 * U)
        # p is 0 before the step: all of it is the update
        got, rate = -weight.double() * m.sign(), opt.lr / (1 - b1 ** t)
        assert torch.isfinite(weight).all() and (got[m == 0] == 0).all()
        worst = torch.stack([(rate * least - got).max(), (got - rate * most).max()])
        assert (got >= rate * least)[m != 0].all() and (got <= rate * most)[m != 0].all(), worst


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", ["fp32", "master", "fp32 and bf16"])
@pytest.mark.parametrize("eps,size", [(1e-30, 1e-20), (1e-30, 3e-19), (1e-30, 1e-12), (1e-30, 1e18), (TINY, 1e-20),
                                      (TINY, 1e-18), (1e-15, 1e-19), (1e-12, 1e-18), (FLUSH / 1.001, 2e-18),
                                      (FLUSH * 1.001, 2e-18), (FLUSH * 1.001, 1e18), (1e-8, 1e-18), (1e-8, 1.0)])
def test_small_eps_and_gradients(gpu_lib, eps, size, kind, bits):
    n = 4096 + 77
    gen = torch.Generator(device="cuda").manual_seed(0)
    g = size * (1 + torch.rand(n, generator=gen, device="cuda")) * (1 - 2 * torch.randint(0, 2, (n,), generator=gen, device="cuda"))
    g[:40] = 0  # of a row that was never touched
    g = g.bfloat16() if kind == "fp32 and bf16" else g
    p = torch.zeros(n, device="cuda", dtype=torch.bfloat16 if kind == "master" else torch.float32)
    opt = gpu_lib.ShardedAdamW([p], lr=1.0, eps=eps, bits=bits, master=kind == "master" or None, seed=5)
    check(opt, g, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_small_eps_with_the_step_on_the_device(gpu_lib, bits):
    g = torch.full((1000,), 1e-19, device="cuda")
    g[:40] = 0
    for eps in (TINY, FLUSH / 1.001, FLUSH * 1.001):
        opt = gpu_lib.ShardedAdamW([torch.zeros(1000, device="cuda")], lr=1.0, eps=eps, bits=bits, capturable=True)
        check(opt, g, 2)


@pytest.mark.gpu
def test_the_class_passes_the_refusals_on(gpu_lib):
    x = torch.zeros(64, device="cuda")
    for kw in (dict(eps=1e-39), dict(lr=1e39), dict(max_norm=1e-50), dict(weight_decay=1e39)):
        opt = gpu_lib.ShardedAdamW([x], **kw)
        with pytest.raises(gpu_lib.TpmlpError) as e:
            opt.step([torch.ones_like(x)])
        assert e.value.status == INVALID and opt.steps == 0 and (x == 0).all()
