"""Argument checks of the operators around the GEMM launches of a step, and their references, without a GPU: no kernel
is launched here."""
import ctypes

import pytest
import torch

import megatron_tensor_transformer_column_gb300 as tp
import step_reference as ref

FAKE = 1 << 20  # never dereferenced
INVALID, SHAPE, ALIGN, UNSUPPORTED, CUDA = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    from megatron_tensor_transformer_column_gb300 import _build
    _build.build()
    return tp.load()


def status_of(call):
    with pytest.raises(tp.TpmlpError) as e:
        call()
    return e.value.status


# ---------------------------------------------------------------- the tokens' norm

@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_reference_gradient_against_differences(kind):
    gen = torch.Generator().manual_seed(0)
    x, dy, ds, v = (torch.randn(3, 24, generator=gen, dtype=torch.float64) for _ in range(4))
    g, b, w = (torch.randn(24, generator=gen, dtype=torch.float64) for _ in range(3))
    f = lambda x, g, b: (ref.norm_forward(x, g, b, kind, 1e-3)[0] * dy).sum() + (x * ds).sum()
    _, mu, r = ref.norm_forward(x, g, b, kind, 1e-3)
    dx, dg, db = ref.norm_backward(x, mu, r, dy, ds, g, kind)
    h = 1e-6
    assert abs((f(x + h * v, g, b) - f(x - h * v, g, b)) / (2 * h) - (dx * v).sum()) < 1e-7
    assert abs((f(x, g + h * w, b) - f(x, g - h * w, b)) / (2 * h) - (dg * w).sum()) < 1e-7
    assert abs((f(x, g, b + h * w) - f(x, g, b - h * w)) / (2 * h) - (db * w).sum()) < 1e-7


def norm_fwd(rows=4, cols=64, kind="layer", dtype="bf16", eps=1e-5, **kw):
    a = {"x": FAKE, "ldx": cols, "residual": None, "ldr": cols, "gain": None, "bias": None, "sum": None, "lds": cols,
         "y": 2 * FAKE, "ldy": cols, "stats": None} | kw
    tp.tpmlp_norm_forward(tp.NormDesc(rows, cols, kind, dtype, eps), *a.values(), stream=0)


def norm_bwd(rows=4, cols=64, kind="layer", dtype="bf16", eps=1e-5, **kw):
    a = {"x": FAKE, "ldx": cols, "stats": 3 * FAKE, "gain": None, "dy": 4 * FAKE, "lddy": cols, "dsum": None,
         "ldds": cols, "dx": 5 * FAKE, "lddx": cols, "dgain": None, "dbias": None, "workspace": None} | kw
    tp.tpmlp_norm_backward(tp.NormDesc(rows, cols, kind, dtype, eps), *a.values(), stream=0)


@pytest.mark.parametrize("call", [norm_fwd, norm_bwd])
def test_norm_descriptions(lib, call):
    assert status_of(lambda: call(kind=2)) == INVALID
    assert status_of(lambda: call(dtype=2)) == INVALID
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert status_of(lambda: call(eps=eps)) == INVALID
    assert status_of(lambda: call(rows=-1)) == SHAPE
    assert status_of(lambda: call(cols=0)) == SHAPE
    assert status_of(lambda: call(cols=60)) == ALIGN
    assert status_of(lambda: call(cols=62, dtype="fp32")) == ALIGN
    assert status_of(lambda: call(cols=16392)) == UNSUPPORTED
    assert status_of(lambda: call(ldx=56)) == SHAPE
    assert status_of(lambda: call(ldx=68)) == ALIGN
    assert status_of(lambda: call(rows=1 << 40, ldx=1 << 20)) == UNSUPPORTED
    assert status_of(lambda: call(x=None)) == INVALID
    assert status_of(lambda: call(x=FAKE + 8)) == ALIGN
    assert lib.tpmlp_norm_forward(None, *[0] * 12) == INVALID  # no desc at all
    if not torch.cuda.is_available():
        assert status_of(call) == CUDA  # the arguments are good


def test_norm_forward_refusals(lib):
    assert status_of(lambda: norm_fwd(y=None)) == INVALID
    assert status_of(lambda: norm_fwd(residual=3 * FAKE)) == INVALID  # no sum
    assert status_of(lambda: norm_fwd(sum=3 * FAKE)) == INVALID      # no residual
    assert status_of(lambda: norm_fwd(residual=3 * FAKE, sum=2 * FAKE)) == INVALID  # sum is y
    assert status_of(lambda: norm_fwd(y=FAKE + 16)) == INVALID  # y overlaps x
    assert status_of(lambda: norm_fwd(y=FAKE, ldy=72)) == INVALID  # in place with another stride
    assert status_of(lambda: norm_fwd(ldx=128, y=FAKE + 112, ldy=128)) == INVALID  # columns in common
    assert status_of(lambda: norm_fwd(gain=2 * FAKE)) == INVALID
    assert status_of(lambda: norm_fwd(stats=2 * FAKE + 256)) == INVALID
    assert status_of(lambda: norm_fwd(stats=FAKE)) == INVALID
    assert status_of(lambda: norm_fwd(gain=3 * FAKE, stats=3 * FAKE)) == INVALID
    assert status_of(lambda: norm_fwd(gain=3 * FAKE + 2)) == ALIGN
    norm_fwd(rows=0, x=None, y=None)


def test_norm_backward_refusals(lib):
    for name in ("stats", "dy", "dx"):
        assert status_of(lambda: norm_bwd(**{name: None})) == INVALID
    assert status_of(lambda: norm_bwd(dgain=6 * FAKE)) == INVALID  # no workspace
    ws = 8 * FAKE
    assert status_of(lambda: norm_bwd(dgain=6 * FAKE, dbias=6 * FAKE, workspace=ws)) == INVALID
    assert status_of(lambda: norm_bwd(dgain=5 * FAKE, workspace=ws)) == INVALID  # dgain in dx
    assert status_of(lambda: norm_bwd(dgain=ws, workspace=ws)) == INVALID
    assert status_of(lambda: norm_bwd(dgain=6 * FAKE, workspace=4 * FAKE)) == INVALID  # the workspace in dy
    assert status_of(lambda: norm_bwd(dx=3 * FAKE)) == INVALID  # dx in stats
    assert status_of(lambda: norm_bwd(dx=4 * FAKE + 128)) == INVALID
    norm_bwd(rows=0, x=None, stats=None, dy=None, dx=None)


def test_norm_workspace(lib):
    size = tp.tpmlp_norm_workspace_size
    assert size(tp.NormDesc(5, 64)) == 5 * 2 * 64 * 4
    assert size(tp.NormDesc(100000, 64)) == size(tp.NormDesc(160, 64)) == 160 * 2 * 64 * 4
    assert size(tp.NormDesc(5, 60)) == size(tp.NormDesc(5, 16392)) == 0
    small = torch.empty(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="smaller"):
        norm_bwd(dgain=6 * FAKE, workspace=small)
    with pytest.raises(ValueError):
        tp.TokenNorm(4, 60)


# ---------------------------------------------------------------- the residual in the epilogue

def row_call(plan, **kw):
    a = {"W2": [FAKE], "b2": None, "residual": 2 * FAKE, "H": [3 * FAKE], "Y": 4 * FAKE, "workspace": 5 * FAKE} | kw
    tp.tpmlp_forward_row_residual(plan, *a.values(), stream=0)


def out_call(plan, **kw):
    a = {"WO": [FAKE], "O": [3 * FAKE], "residual": 2 * FAKE, "Z": 4 * FAKE, "workspace": 5 * FAKE} | kw
    tp.tpmlp_attn_out_forward_residual(plan, *a.values(), stream=0)


def block_call(fn, plan, **kw):
    a = {"X": 6 * FAKE, "W1": [FAKE], "W3": None, "W2": [FAKE], "b1": None, "b3": None, "b2": None,
         "residual": 2 * FAKE, "Y": 4 * FAKE, "kept": [7 * FAKE], "H": [3 * FAKE], "workspace": 5 * FAKE} | kw
    fn(plan, *a.values(), stream=0)


def test_residual_refusals(lib):
    """Without a GPU the first thing that is missed is the device; with one, the argument."""
    if torch.cuda.is_available():
        pytest.skip("the calls without a device")
    mlp, proj = tp.Plan(64, 64, [64]), tp.AttnPlan(64, 64, [64], [64])
    calls = [lambda p, **kw: row_call(p, **kw)]
    calls += [lambda p, f=f, **kw: block_call(f, p, **kw) for f in (tp.tpmlp_forward_residual,
                                                                     tp.tpmlp_forward_ckpt8_residual)]
    for call in calls:
        assert status_of(lambda: call(mlp)) == CUDA
        assert status_of(lambda: call(proj)) == INVALID
        with pytest.raises(ValueError, match="expected 1"):
            call(mlp, W2=[])
    assert status_of(lambda: out_call(proj)) == CUDA
    assert status_of(lambda: out_call(mlp)) == INVALID
    assert status_of(lambda: out_call(proj, workspace=None)) == INVALID


@pytest.mark.gpu
def test_residual_refusals_with_a_device(gpu_lib):
    mlp, proj = tp.Plan(64, 64, [64]), tp.AttnPlan(64, 64, [64], [64])
    fns = [lambda **kw: row_call(mlp, **kw)]
    fns += [lambda f=f, **kw: block_call(f, mlp, **kw) for f in (tp.tpmlp_forward_residual,
                                                                  tp.tpmlp_forward_ckpt8_residual)]
    for call, out in [(c, "Y") for c in fns] + [(lambda **kw: out_call(proj, **kw), "Z")]:
        assert status_of(lambda: call(residual=None)) == INVALID
        assert status_of(lambda: call(residual=2 * FAKE + 8)) == ALIGN
        assert status_of(lambda: call(residual=4 * FAKE + 16)) == INVALID  # overlaps the output
        assert status_of(lambda: call(residual=4 * FAKE - 8176)) == INVALID
        assert status_of(lambda: call(**{out: None})) == INVALID
    m = tp.ShardedMLP(64, 64, [64])
    x = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x[:32], x.t()):
        with pytest.raises(ValueError, match="residual"):
            m.row_forward([x], [x], residual=bad)
        with pytest.raises(ValueError, match="residual"):
            m.forward(x, [x], [x], residual=bad)


# ---------------------------------------------------------------- AdamW and the norm of the gradients

ODD = [5, 0, 300]


def step_call(sizes=(512, 100), dtype="bf16", grad_dtype=None, bits=32, hyper=None, norm=None, **kw):
    n = len(sizes)
    at = lambda base: [base * FAKE + (1 << 12) * k for k in range(n)]
    a = {"p": at(1), "g": at(2), "master": None, "m": at(3), "v": at(4), "weight_decay": None} | kw
    tp.tpmlp_adamw_step(tp.AdamWDesc(sizes, dtype, grad_dtype, bits), *a.values(),
                        tp.AdamWHyper(**(hyper or {})), norm, stream=0)


def norm_call(sizes=(512, 100), **kw):
    a = {"g": [FAKE, 2 * FAKE], "norm": 3 * FAKE, "workspace": 4 * FAKE} | kw
    tp.tpmlp_grad_norm(tp.AdamWDesc(sizes), *a.values(), stream=0)


def test_adamw_sizes(lib):
    assert [tp.tpmlp_adamw_state_size(32, n) for n in (0, 1, 1000)] == [0, 4, 4000]
    assert [tp.tpmlp_adamw_state_size(8, n) for n in (0, 1, 256, 257)] == [0, 257, 257, 514]
    assert tp.tpmlp_adamw_state_size(8, -1) == tp.tpmlp_adamw_state_size(16, 8) == tp.tpmlp_adamw_state_size(8, 1 << 50) == 0
    assert tp.tpmlp_grad_norm_workspace_size() == 256 + 8 * 1281


def test_adamw_descriptions(lib):
    for kw in (dict(dtype=2), dict(grad_dtype=5), dict(bits=16), dict(p=None), dict(p=[FAKE, 0]), dict(m=None),
               dict(v=[0, FAKE]), dict(dtype="fp32", master=[5 * FAKE, 6 * FAKE]),
               dict(weight_decay=[0.1, float("nan")])):
        assert status_of(lambda: step_call(**kw)) == INVALID
    assert status_of(lambda: step_call(sizes=(-1, 3))) == SHAPE
    assert status_of(lambda: step_call(sizes=(1 << 41, 3))) == SHAPE
    for name in ("p", "g", "m", "v", "master"):
        assert status_of(lambda: step_call(**{name: [FAKE * 8, FAKE * 9 + 8]})) == ALIGN
    with pytest.raises(ValueError, match="expected 2"):
        step_call(g=[FAKE])
    with pytest.raises(ValueError, match="expected 2"):
        step_call(weight_decay=[0.1])
    nan, inf = float("nan"), float("inf")
    for h in (dict(lr=nan), dict(lr=inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=nan), dict(eps=0.0), dict(eps=nan),
              dict(eps=inf), dict(grad_scale=inf), dict(grad_scale=-1.0), dict(max_norm=-1.0), dict(max_norm=nan), dict(max_norm=1.0),
              dict(step=0), dict(step=-3)):
        assert status_of(lambda: step_call(hyper=h)) == INVALID
    assert status_of(lambda: step_call(hyper=dict(step_device=8 * FAKE + 4))) == ALIGN
    assert status_of(lambda: step_call(hyper=dict(lr_device=8 * FAKE + 2))) == ALIGN
    assert status_of(lambda: step_call(norm=8 * FAKE + 2)) == ALIGN
    assert lib.tpmlp_adamw_step(None, *[None] * 9) == INVALID
    if not torch.cuda.is_available():
        for kw in ({}, dict(bits=8), dict(master=[5 * FAKE, 6 * FAKE]), dict(norm=8 * FAKE, hyper=dict(max_norm=1.0))):
            assert status_of(lambda: step_call(**kw)) == CUDA  # the arguments are good
        assert status_of(norm_call) == CUDA


def test_adamw_overlaps(lib):
    assert status_of(lambda: step_call(p=[FAKE, FAKE])) == INVALID  # one tensor twice
    assert status_of(lambda: step_call(p=[FAKE, FAKE + 1008])) == INVALID  # 512 bf16 end at 1024
    assert status_of(lambda: step_call(g=[FAKE, 9 * FAKE])) == INVALID  # a gradient that is a parameter
    assert status_of(lambda: step_call(v=[3 * FAKE, 9 * FAKE])) == INVALID  # m is v
    assert status_of(lambda: step_call(bits=8, m=[9 * FAKE, 9 * FAKE + 512])) == INVALID  # 514 bytes
    assert status_of(lambda: step_call(master=[FAKE + 512, 9 * FAKE])) == INVALID
    assert status_of(lambda: step_call(norm=4 * FAKE)) == INVALID
    assert status_of(lambda: step_call(hyper=dict(lr_device=FAKE + 4))) == INVALID
    assert status_of(lambda: step_call(hyper=dict(step_device=3 * FAKE))) == INVALID
    if not torch.cuda.is_available():
        assert status_of(lambda: step_call(g=[9 * FAKE, 9 * FAKE])) == CUDA  # one gradient for two tensors
        assert status_of(lambda: step_call(p=[FAKE, FAKE + 1024])) == CUDA


def test_grad_norm_refusals(lib):
    assert status_of(lambda: norm_call(g=None)) == INVALID
    assert status_of(lambda: norm_call(norm=None)) == INVALID
    assert status_of(lambda: norm_call(workspace=None)) == INVALID
    assert status_of(lambda: norm_call(norm=3 * FAKE + 2)) == ALIGN
    assert status_of(lambda: norm_call(g=[FAKE, 2 * FAKE + 2])) == ALIGN
    assert status_of(lambda: norm_call(norm=FAKE + 4)) == INVALID
    assert status_of(lambda: norm_call(workspace=2 * FAKE)) == INVALID
    assert status_of(lambda: norm_call(norm=4 * FAKE + 256)) == INVALID  # inside the workspace


def test_unpack_refusals(lib):
    call = lambda bits=8, m=[FAKE], v=[2 * FAKE], mo=[3 * FAKE], vo=[4 * FAKE]: tp.tpmlp_adamw8_unpack(
        tp.AdamWDesc([300], bits=bits), m, v, mo, vo, stream=0)
    assert status_of(lambda: call(bits=32)) == INVALID
    assert status_of(lambda: call(m=None)) == INVALID
    assert status_of(lambda: call(mo=[FAKE])) == INVALID
    assert status_of(lambda: call(mo=[2 * FAKE - 16])) == INVALID
    assert status_of(lambda: call(mo=[4 * FAKE])) == INVALID
    assert status_of(lambda: call(mo=[3 * FAKE + 2])) == ALIGN
    call(m=None, mo=None, v=None, vo=None)


def test_adamw_reference_rounding():
    """Random bits that cover every value give the value back in the mean; the codes' own values stay."""
    e = torch.tensor([3])
    grid = torch.arange(0, 65536, 256)[None]
    for second in (False, True):
        least = 1.125 * 2.0 ** (3 - (31 if second else 15))
        for y in (1.0, 1.3, 9.999, 0.77, 3 * least) + (() if second else (0.3 * least,)):
            x = torch.full((1, 256), y, dtype=torch.float64)
            kept = ref.rounded(x, e, grid, second)
            step = 2.0 ** (torch.frexp(torch.tensor(max(y, least)))[1].item() - 4)
            assert abs(kept.mean().item() - y) <= max(step, least) / 128
    v = ref.values(torch.cat([torch.arange(256, dtype=torch.uint8), torch.tensor([91], dtype=torch.uint8)]), 256, True)[0]
    assert (v[1:] > v[:-1]).all() and v[255] == 1.875 and v[1] == 1.125 * 2.0 ** -31
    assert torch.equal(ref.rounded(v[None], torch.tensor([0]), torch.full((1, 256), 65535), True)[0], v)


def test_adamw_reference_hash():
    """Known values of the hash, worked out with Python's integers."""
    def h(x):
        x = ((x ^ (x >> 16)) * 0x7feb352d) % 2 ** 32
        x = ((x ^ (x >> 15)) * 0x846ca68b) % 2 ** 32
        return x ^ (x >> 16)
    key = h(h(h(h(5) ^ 7) ^ 9) ^ 0)
    a = h(h(key ^ 2) ^ 1)
    r = ref.randoms((7 << 32) + 5, 9, (1 << 32) + 2, 1)[0]
    assert r[100].item() == h((a + 50 * 0x9e3779b9) % 2 ** 32) & 0xffff
    assert r[101].item() == h((a + 50 * 0x9e3779b9) % 2 ** 32) >> 16


def test_adamw_reference_against_the_gradient_of_a_quadratic():
    """Minimising x^2 / 2 moves x towards 0 by lr a step at first (the corrections at work)."""
    x, m, v = torch.tensor([2.0, -3.0]).double(), torch.zeros(2), torch.zeros(2)
    for t in (1, 2, 3):
        y, m, v = ref.adamw(x, x, m, v, t, 1e-3, 0.9, 0.999, 1e-12, 0.0)
        assert torch.allclose((x - y).abs(), torch.full((2,), 1e-3, dtype=torch.float64), rtol=1e-2)
        x = y
