"""Calls of the head norm with rotation and of the 8-bit checkpoints that need no GPU: what is accepted, what is
refused, and what the Python layer keeps."""
import copy
import ctypes
import pickle

import pytest
import torch

import megatron_tensor_transformer_column_gb300 as tp

A = 1 << 24  # addresses that are never dereferenced


@pytest.fixture(scope="module")
def lib():
    from megatron_tensor_transformer_column_gb300 import _build
    _build.build()
    return tp.load()


def status_of(call):
    with pytest.raises(tp.TpmlpError) as e:
        call()
    return e.value.status


def heads_plan(T, norm=True, dtype="bf16"):
    p = tp.AttnPlan(T, 64, [128, 64], [64, 64], dtype)
    tp.tpmlp_attn_plan_set_qk_norm_rope(p, 64, norm=norm)
    return p


def test_backward_of_the_rotation_alone_takes_no_x(lib):
    """QKV may be missing in the backward call without a norm, and in no other (no tokens: nothing is launched)."""
    n = [None, None]
    tp.tpmlp_attn_qk_norm_rope_backward(heads_plan(0, False), None, None, None, None, n, n, n, None, None, None, stream=0)
    assert status_of(lambda: tp.tpmlp_attn_qk_norm_rope_backward(heads_plan(0), None, None, None, None, n, n, n, None,
                                                                 None, None, stream=0)) == 1
    assert status_of(lambda: tp.tpmlp_attn_qk_norm_rope_forward(heads_plan(0, False), None, None, None, None, n,
                                                                stream=0)) == 1
    # what is given is still looked at
    far = [A + (i << 22) for i in range(8)]
    p = heads_plan(16, False)
    call = lambda **kw: tp.tpmlp_attn_qk_norm_rope_backward(
        p, *{**dict(QKV=None, pos=None, gq=None, gk=None, dQK=far[:2], dV=far[2:4], dQKV=far[4:6], dgq=None, dgk=None,
                    workspace=None), **kw}.values(), stream=0)
    assert status_of(lambda: call(QKV=[far[6], None])) == 1
    assert status_of(lambda: call(QKV=[far[6], far[4]])) == 1       # over an output
    assert status_of(lambda: call(QKV=[far[6] + 8, far[7]])) == 3
    assert status_of(lambda: call(dQK=[far[0], far[4]])) == 1       # another shard's output
    assert status_of(lambda: call(dQK=[far[0], None])) == 1


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_describing_the_heads_keeps_the_workspace(lib, dtype):
    """Kernels in flight and captured graphs hold its address, and its status word."""
    proj = tp.ShardedAttentionProj(16, 64, [256], [256], dtype, device="cpu")
    ws, at = proj.workspace, proj.workspace.data_ptr()
    for D in (2, 64, 256):
        proj.set_qk_norm_rope(D)
        assert proj.workspace is ws and ws.data_ptr() == at and ws.numel() >= tp.tpmlp_workspace_size(proj.plan)


@pytest.mark.parametrize("name", ["TPMLPFunction", "TPMLPCheckpointFunction"])
def test_autograd_functions_can_be_copied_and_pickled(name):
    fn = getattr(tp, name)
    for used in (False, True):
        if used:
            assert fn.__name__ == name
        for other in (copy.copy(fn), copy.deepcopy(fn), copy.deepcopy([fn])[0], pickle.loads(pickle.dumps(fn))):
            assert other.__name__ == name and other.apply == fn.apply
    assert tp.TPMLPFunction.__name__ != tp.TPMLPCheckpointFunction.__name__


@pytest.mark.parametrize("element", [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int64])
def test_arrays_of_addresses_of_any_integer_type(lib, element):
    """A ctypes array counts as a sequence of addresses, whatever its elements' type."""
    both = lambda *xs: (element * 2)(*xs)
    n = both(0, 0)
    p = heads_plan(0)  # no tokens: accepted, and nothing is launched
    tp.tpmlp_attn_qk_norm_rope_forward(p, n, None, None, None, n, stream=0)
    p = heads_plan(16)
    call = lambda QK: tp.tpmlp_attn_qk_norm_rope_forward(p, both(A, A + (1 << 22)), None, None, None, QK, stream=0)
    assert status_of(lambda: call(both(A + (1 << 24), A + (1 << 26) + 8))) == 3
    assert status_of(lambda: call(both(A + (1 << 24), 0))) == 1
    m = tp.AttnPlan(16, 64, [128, 64], [64, 64])
    with pytest.raises(tp.TpmlpError):  # a misaligned entry, or no device
        tp.tpmlp_attn_qkv_forward(m, A, both(A + 8, A + 8), both(A, A), A, stream=0)


def test_lists_shorter_than_the_shards_are_refused(lib):
    """The library would read addresses past the end of the host array."""
    p, n = heads_plan(0), [None, None]
    fwd = dict(QKV=n, pos=None, gq=None, gk=None, QK=n)
    bwd = dict(QKV=n, pos=None, gq=None, gk=None, dQK=n, dV=n, dQKV=n, dgq=None, dgk=None, workspace=None)
    calls = [(tp.tpmlp_attn_qk_norm_rope_forward, p, fwd), (tp.tpmlp_attn_qk_norm_rope_backward, p, bwd)]
    for act in ("gelu", "swiglu"):
        m, sw = tp.Plan(0, 64, [64, 32], act), act == "swiglu"
        a, w, w3 = [None] * (4 if sw else 2), [A, A], [A, A] if sw else None
        calls += [(tp.tpmlp_forward_ckpt8, m, dict(X=None, W1=w, W3=w3, W2=w, b1=w, b3=w3, b2=None, Y=None, ckpt=a, H=n,
                                                   workspace=A)),
                  (tp.tpmlp_backward_ckpt8, m, dict(X=None, W1=w, W3=w3, W2=w, ckpt=a, H=n, dY=None, dact=a, dX=None,
                                                    dW1=w, dW3=w3, dW2=w, db1=w, db3=w3, db2=None, workspace=A))]
    for f, plan, args in calls:
        for name, xs in args.items():
            if not isinstance(xs, list):
                continue
            for short in (xs[:-1], (ctypes.c_void_p * (len(xs) - 1))()):
                with pytest.raises(ValueError):
                    f(plan, *{**args, name: short}.values(), stream=0)
    for f, plan, args in calls[:2]:  # whole ones, and longer ones, are taken
        f(plan, *args.values(), stream=0)
        f(plan, *{**args, "QKV": [None] * 3}.values(), stream=0)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_checkpoint_function_refuses_what_it_would_leave_out(lib, act):
    """Biases behind the weights, or W3 with GeLU: the forward pass ignored them."""
    mlp = tp.ShardedMLP(8, 16, [16, 8], act, device="cpu")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    ws = [z(16, 16), z(16, 8), z(16, 16), z(8, 16)] + ([z(16, 16), z(16, 8)] if act == "swiglu" else [])
    for weights in (ws + [z(16), z(8)], ws[:-1], ws[:2], []):
        with pytest.raises(ValueError, match="weights"):
            tp.TPMLPCheckpointFunction.apply(mlp, z(8, 16), *weights)
