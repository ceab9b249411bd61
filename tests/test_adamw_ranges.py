"""AdamW at the ends of the fp32 range: numbers that it does not hold are refused."""
import pytest
import torch

import megatron_tensor_transformer_column_gb300 as tp
from test_step_operators_cpu import CUDA, FAKE, INVALID, status_of, step_call

TINY = 2.0 ** -126


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


@pytest.mark.gpu
def test_the_class_passes_the_refusals_on(gpu_lib):
    x = torch.zeros(64, device="cuda")
    for kw in (dict(eps=1e-39), dict(lr=1e39), dict(max_norm=1e-50), dict(weight_decay=1e39)):
        opt = gpu_lib.ShardedAdamW([x], **kw)
        with pytest.raises(gpu_lib.TpmlpError) as e:
            opt.step([torch.ones_like(x)])
        assert e.value.status == INVALID and opt.steps == 0 and (x == 0).all()
