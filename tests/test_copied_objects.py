"""Copies and pickles of the classes work on memory of their own, or are refused."""
import contextlib
import copy
import gc
import pickle
import types

import pytest
import torch

import megatron_tensor_transformer_column_gb300 as tp

COPIES = [copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))]


@pytest.fixture(scope="module")
def lib():
    from megatron_tensor_transformer_column_gb300 import _build
    _build.build()
    return tp.load()


@pytest.mark.parametrize("how", COPIES, ids=["deepcopy", "pickle"])
def test_a_copied_norm_hands_over_its_own_workspace(lib, monkeypatch, how):
    """Without a GPU: the addresses that the calls get."""
    norm = tp.TokenNorm(4, 64, device="cpu")
    other = how(norm)
    calls = []
    fake = types.SimpleNamespace(tpmlp_norm_forward=lambda *a: calls.append(a) or 0,
                                 tpmlp_norm_backward=lambda *a: calls.append(a) or 0)
    monkeypatch.setattr(tp, "_lib", None)  # as in a process that has only read the pickle
    monkeypatch.setattr(tp, "load", lambda: fake)
    monkeypatch.setattr(tp, "_on", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(tp, "_current", lambda *a: 0)
    x, g = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for n in (other, norm):
        y, stats, s = n.forward(x, g)
        n.backward(s, stats, x, g)
        assert calls[-1][13] == n.workspace.data_ptr()
    assert norm.workspace.data_ptr() != other.workspace.data_ptr()
    assert bytes(norm.desc) == bytes(other.desc) and other.device == other.workspace.device


@pytest.mark.gpu
@pytest.mark.parametrize("how", COPIES, ids=["deepcopy", "pickle"])
def test_a_copied_norm_outlives_the_original(gpu_lib, how):
    """The copy's gradients, and the memory that was the original's workspace."""
    T, d = 700, 512
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, dy, ds = (torch.randn(T, d, generator=gen, device="cuda").bfloat16() for _ in range(3))
    g = torch.randn(d, generator=gen, device="cuda").bfloat16()
    norm = gpu_lib.TokenNorm(T, d, "layer", "bf16")
    y, stats, s = norm.forward(x, g, g)
    want = norm.backward(s, stats, dy, g, dsum=ds, bias_grad=True)
    other = how(norm)
    old = norm.workspace
    del norm
    gc.collect()
    old.fill_(7)
    got = other.backward(s, stats, dy, g, dsum=ds, bias_grad=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(other.forward(x, g, g)[0], y)
    assert (old == 7).all()


@pytest.mark.parametrize("make", [lambda: tp.ShardedMLP(8, 64, [64], device="cpu"),
                                  lambda: tp.ShardedAttentionProj(8, 64, [64], [64], device="cpu")])
def test_classes_that_hold_a_plan_refuse(lib, make):
    x = make()
    for how in COPIES:
        with pytest.raises(Exception, match="pickle"):
            how(x)


@pytest.mark.gpu
def test_the_optimizer_refuses(gpu_lib):
    opt = gpu_lib.ShardedAdamW([torch.zeros(8, device="cuda")])
    for how in COPIES:
        with pytest.raises(Exception, match="pickle"):
            how(opt)
