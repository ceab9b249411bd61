"""A step is an in-place change of the weights for autograd: a graph that still needs the old ones refuses."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
def test_an_older_graph_refuses(gpu_lib, bits, capturable):
    w = torch.randn(64, 32, device="cuda", requires_grad=True)
    v = torch.randn(32, 8, device="cuda", requires_grad=True)
    x = torch.randn(16, 64, device="cuda")
    opt = gpu_lib.ShardedAdamW([w, v], lr=1e-2, bits=bits, capturable=capturable)
    y = ((x @ w) @ v).square().sum()
    y.backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()  # needs the old v
    ((x @ w) @ v).square().sum().backward()  # a new one does not mind
    opt.step()


def test_the_blocks_functions_refuse_too(gpu_lib):
    mlp = gpu_lib.ShardedMLP(64, 64, [64, 64])
    bf = lambda *s: (0.1 * torch.randn(*s, device="cuda")).bfloat16()
    ws = [bf(64, 64).requires_grad_() for _ in range(4)]
    x = bf(64, 64).requires_grad_()
    opt = gpu_lib.ShardedAdamW(ws, lr=1e-2, master=True)
    for fn, args in ((gpu_lib.TPMLPFunction, (x,)), (gpu_lib.TPMLPCheckpointFunction, (x,)),
                     (gpu_lib.TPMLPResidualFunction, (x, x))):
        y = fn.apply(mlp, *args, *ws).float().sum()
        y.backward(retain_graph=True)
        opt.step()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        for w in ws:
            w.grad = None


def test_a_refused_step_changes_no_version(gpu_lib):
    w = torch.randn(64, device="cuda", requires_grad=True)
    opt = gpu_lib.ShardedAdamW([w])
    n = w._version
    with pytest.raises(gpu_lib.TpmlpError):
        opt.step([w.detach()])
    assert w._version == n
    opt.step([torch.ones_like(w)])
    assert w._version > n


def test_weights_made_under_inference_mode(gpu_lib):
    with torch.inference_mode():
        w = torch.ones(64, device="cuda")
        opt = gpu_lib.ShardedAdamW([w])
        opt.step([torch.ones(64, device="cuda")])
    assert (w != 1).all()
