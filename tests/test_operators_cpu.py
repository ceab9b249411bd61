"""Argument checks of the norm with rotation and of the 8-bit checkpoints, and their references, without a GPU: no
kernel is launched here."""
import ctypes

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_column_gb300 as tp
import operators_reference as ref

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from megatron_tensor_transformer_column_gb300 import _build
    _build.build()
    return tp.load()


def status_of(call):
    with pytest.raises(tp.TpmlpError) as e:
        call()
    return e.value.status


# ---------------------------------------------------------------- the references themselves

@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("norm", [True, False])
def test_reference_gradient_against_differences(layout, norm):
    rng = np.random.default_rng(0)
    x, dy, g = rng.normal(size=(3, 2, 12)), rng.normal(size=(3, 2, 12)), rng.normal(size=12)
    pos, freq = np.array([0, 7, -3]), ref.frequencies(8)
    f = lambda x, g: (ref.heads_forward(x, pos, freq, layout, g if norm else 1.0, 1e-3, norm)[0] * dy).sum()
    dx, dg = ref.heads_backward(x, dy, pos, freq, layout, g, 1e-3, norm)[:2]
    v, w, h = rng.normal(size=x.shape), rng.normal(size=g.shape), 1e-6
    assert abs((f(x + h * v, g) - f(x - h * v, g)) / (2 * h) - (dx * v).sum()) < 1e-7
    if norm:
        assert abs((f(x, g + h * w) - f(x, g - h * w)) / (2 * h) - (dg * w).sum()) < 1e-7


def test_reference_codes():
    """The table against torch's own e4m3 type, and the rounding against its conversion."""
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), ref.E4M3)
    v = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.05, 0.05, 20001)])
    assert np.array_equal(ref.encode(v.double().numpy()), v.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_pack_bound():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(40, 50)) * np.exp(4 * rng.normal(size=50))
    codes, scale = ref.pack(x)
    v = ref.values(codes, scale, 50)
    step = np.repeat(2.0 ** (scale.astype(float) - 127 - 10), 16, 1)[:, :50]
    assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step)).all()


# ---------------------------------------------------------------- refusals

@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=64), 0), (dict(head_dim=32, rotary_dim=0), 0), (dict(head_dim=64, rotary_dim=6), 0),
    (dict(head_dim=128), 2),                    # dkv_i = 64 is not a whole number of heads
    (dict(head_dim=0), 2), (dict(head_dim=-2), 2), (dict(head_dim=1, rotary_dim=0), 2),
    (dict(head_dim=64, rotary_dim=66), 2), (dict(head_dim=64, rotary_dim=3), 2), (dict(head_dim=64, rotary_dim=-2), 2),
    (dict(head_dim=512), 4),
    (dict(head_dim=64, layout=2), 1), (dict(head_dim=64, norm=2), 1),
    (dict(head_dim=64, eps=0.0), 1), (dict(head_dim=64, eps=-1.0), 1), (dict(head_dim=64, eps=float("nan")), 1),
    (dict(head_dim=64, eps=float("inf")), 1), (dict(head_dim=64, base=0.0), 1),
    (dict(head_dim=64, base=float("inf")), 1), (dict(head_dim=64, inv_freq=[float("nan")] * 32), 1),
    (dict(head_dim=64, eps=0.0, norm=False), 0), (dict(head_dim=64, base=0.0, inv_freq=[1.0] * 32), 0),
])
def test_head_description(lib, kw, status):
    p = tp.AttnPlan(16, 64, [128], [64])
    if status == 0:
        tp.tpmlp_attn_plan_set_qk_norm_rope(p, **kw)
    else:
        assert status_of(lambda: tp.tpmlp_attn_plan_set_qk_norm_rope(p, **kw)) == status


def test_head_description_of_other_plans(lib):
    assert status_of(lambda: tp.tpmlp_attn_plan_set_qk_norm_rope(tp.Plan(16, 64, [64]), 64)) == 1
    assert lib.tpmlp_attn_plan_set_qk_norm_rope(None, None) == 1
    with pytest.raises(ValueError):
        tp.tpmlp_attn_plan_set_qk_norm_rope(tp.AttnPlan(16, 64, [64], [64]), 64, inv_freq=[1.0])


def test_workspace_grows_only_with_the_norm(lib):
    p = tp.AttnPlan(16, 64, [64], [64], "fp32")
    small = tp.tpmlp_workspace_size(p)
    tp.tpmlp_attn_plan_set_qk_norm_rope(p, 64, norm=False)
    assert tp.tpmlp_workspace_size(p) == small == 256
    tp.tpmlp_attn_plan_set_qk_norm_rope(p, 64)
    assert tp.tpmlp_workspace_size(p) == 256 + 4096 * 64 * 4
    b = tp.AttnPlan(16, 64, [64], [64], "bf16")
    n = tp.tpmlp_workspace_size(b)
    tp.tpmlp_attn_plan_set_qk_norm_rope(b, 64)
    assert tp.tpmlp_workspace_size(b) == n and n >= 16384 + 4096 * 256 * 4


def _plan(norm=True, T=16):
    p = tp.AttnPlan(T, 64, [128, 64], [64, 64], "bf16")
    tp.tpmlp_attn_plan_set_qk_norm_rope(p, 64, norm=norm)
    return p


A, B = 1 << 24, 1 << 26  # far enough apart for every buffer here


def fwd(p, QKV=(A, A + (1 << 20)), pos=None, gq=None, gk=None, QK=(B, B + (1 << 20))):
    tp.tpmlp_attn_qk_norm_rope_forward(p, list(QKV), pos, gq, gk, list(QK), stream=0)


def bwd(p, QKV=(A, A + (1 << 20)), pos=None, gq=None, gk=None, dQK=(B, B + (1 << 20)), dV=None,
        dQKV=(2 * B, 2 * B + (1 << 20)), dgq=None, dgk=None, ws=None):
    tp.tpmlp_attn_qk_norm_rope_backward(p, list(QKV), pos, gq, gk, list(dQK), dV, list(dQKV), dgq, dgk, ws, stream=0)


def test_forward_refusals(lib):
    p = _plan()
    assert status_of(lambda: fwd(tp.AttnPlan(16, 64, [128, 64], [64, 64]))) == 1  # heads not described
    assert status_of(lambda: fwd(tp.Plan(16, 64, [64]))) == 1
    assert status_of(lambda: fwd(p, QKV=(A, None))) == 1
    assert status_of(lambda: fwd(p, QK=(None, B))) == 1
    assert status_of(lambda: fwd(p, QKV=(A + 8, A + (1 << 20)))) == 3
    assert status_of(lambda: fwd(p, pos=FAKE + 4)) == 3
    assert status_of(lambda: fwd(p, gq=FAKE + 2)) == 3
    assert status_of(lambda: fwd(_plan(norm=False), gk=FAKE)) == 1
    assert status_of(lambda: fwd(p, QK=(A + 16, B))) == 1            # overlaps its own input without being it
    assert status_of(lambda: fwd(p, QK=(B, A))) == 1                 # another shard's input
    assert status_of(lambda: fwd(p, QK=(A - 16 * 192 * 2 + 16, B))) == 1  # its last bytes reach into QKV[0]
    assert status_of(lambda: fwd(p, QK=(B, B))) == 1                 # two shards' outputs on one another
    assert status_of(lambda: fwd(p, QK=(B, B + 6128))) == 1


def test_backward_refusals(lib):
    p = _plan()
    assert status_of(lambda: bwd(p, dQK=(B, None))) == 1
    assert status_of(lambda: bwd(p, dV=[None, B])) == 1
    assert status_of(lambda: bwd(p, dQKV=(A, 2 * B))) == 1           # over QKV
    assert status_of(lambda: bwd(p, dQKV=(B + 16, 2 * B))) == 1      # over dQK without being it
    assert status_of(lambda: bwd(p, dV=[2 * B + 64, B + (1 << 21)])) == 1
    assert status_of(lambda: bwd(p, dgq=FAKE)) == 1                  # needs a workspace
    assert status_of(lambda: bwd(p, dgq=FAKE, dgk=FAKE, ws=FAKE)) == 1
    assert status_of(lambda: bwd(p, dQKV=(2 * B, 2 * B + 64))) == 1
    assert status_of(lambda: bwd(p, dgk=FAKE + 8, ws=FAKE)) == 3
    assert status_of(lambda: bwd(_plan(norm=False), dgq=FAKE, ws=FAKE)) == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour")
def test_no_cpu_fallback_without_gpu(lib):
    p, m = _plan(), tp.Plan(16, 64, [64], "gelu", "bf16")
    for call in (lambda: fwd(p), lambda: fwd(p, QK=(A, A + (1 << 20))), lambda: bwd(p), lambda: bwd(p, dQK=(2 * B, B)),
                 lambda: tp.tpmlp_ckpt8_pack("bf16", 4, 16, A, 16, B, stream=0),
                 lambda: tp.tpmlp_ckpt8_unpack("fp32", 4, 16, A, B, 16, stream=0),
                 lambda: tp.tpmlp_forward_ckpt8(m, FAKE, [FAKE], None, [FAKE], None, None, None, FAKE, [FAKE], [FAKE],
                                                FAKE, stream=0),
                 lambda: tp.tpmlp_backward_ckpt8(m, FAKE, [FAKE], None, [FAKE], [FAKE], [FAKE], FAKE, [FAKE], FAKE,
                                                 [FAKE], None, [FAKE], None, None, None, FAKE, stream=0)):
        assert status_of(call) in (4, 5)


def test_checkpoint_sizes(lib):
    for rows, cols in ((0, 16), (1, 8), (32, 16), (33, 17), (1000, 1376)):
        assert tp.tpmlp_ckpt8_size(rows, cols) == ref.nbytes(rows, cols)
    assert tp.tpmlp_ckpt8_size(1 << 24, 1 << 16) == (1 << 19) * (1 << 12) * 544
    assert tp.tpmlp_ckpt8_size(-1, 16) == tp.tpmlp_ckpt8_size(16, -1) == tp.tpmlp_ckpt8_size(1 << 31, 1) == 0


@pytest.mark.parametrize("args,status", [
    ((9, 4, 16, A, 16, B), 1), (("bf16", -1, 16, A, 16, B), 2), (("bf16", 4, 0, A, 16, B), 2),
    (("bf16", 4, 16, A, 8, B), 2), (("bf16", 4, 12, A, 16, B), 3), (("bf16", 4, 16, A, 20, B), 3),
    (("fp32", 4, 6, A, 8, B), 3), (("bf16", 1 << 31, 16, A, 16, B), 4), (("bf16", 4, 16, None, 16, B), 1),
    (("bf16", 4, 16, A, 16, None), 1), (("bf16", 4, 16, A + 8, 16, B), 3), (("bf16", 4, 16, A, 16, B + 4), 3),
    (("bf16", 1 << 30, 16, A, 1 << 30, B), 4),
    (("bf16", 4, 16, A, 16, A), 1), (("bf16", 4, 16, A, 1024, A + 3 * 2048 + 16), 1),
])
def test_pack_refusals(lib, args, status):
    dtype, rows, cols, x, ld, ckpt = args
    assert status_of(lambda: tp.tpmlp_ckpt8_pack(dtype, rows, cols, x, ld, ckpt, stream=0)) == status
    assert status_of(lambda: tp.tpmlp_ckpt8_unpack(dtype, rows, cols, ckpt, x, ld, stream=0)) == status


def test_rows_between_a_strided_tensors_may_not_hold_the_checkpoint(lib):
    """Only the bytes past the last row's end count as outside the tensor."""
    assert status_of(lambda: tp.tpmlp_ckpt8_pack("bf16", 4, 16, A, 1024, A + 64, stream=0)) == 1


def test_block_pass_refusals(lib):
    m = tp.Plan(16, 64, [64], "swiglu", "bf16")
    ok = dict(X=FAKE, W1=[FAKE], W3=[FAKE], W2=[FAKE], b1=None, b3=None, b2=None, Y=FAKE, ckpt=[FAKE, FAKE], H=[FAKE],
              workspace=FAKE)
    call = lambda **kw: tp.tpmlp_forward_ckpt8(m, *{**ok, **kw}.values(), stream=0)
    ap = tp.AttnPlan(16, 64, [64], [64])
    assert status_of(lambda: tp.tpmlp_forward_ckpt8(ap, *ok.values(), stream=0)) == 1
    assert status_of(lambda: call(workspace=None)) == 1
    assert status_of(lambda: call(workspace=FAKE + 8)) == 3


def test_python_checks():
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        tp.ckpt8_pack(x)
    with pytest.raises(ValueError):
        tp.ckpt8_unpack(torch.zeros(544, dtype=torch.uint8), 4, 16)
    with pytest.raises(ValueError):
        tp.ckpt8_unpack(torch.zeros(10, dtype=torch.uint8), 4, 16)
    with pytest.raises(ValueError):
        p = _plan()
        tp.tpmlp_attn_qk_norm_rope_forward(p, [A, A], torch.zeros(16, dtype=torch.int32), None, None, [B, B], stream=0)
