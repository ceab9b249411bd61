"""Rotation without a norm (norm = 0): the forward pass at every vector width, and the backward pass, whose result
dx = w (dy rotated back) does not contain x.  Bounds: those of test_gpu_qk_norm_rope."""
import numpy as np
import pytest
import torch

from test_gpu_qk_norm_rope import SHAPES, check, check_backward, check_forward, heads, k_of, make, np64, proj_of, q_of

import operators_reference as ref

pytestmark = pytest.mark.gpu


def shape(tp, T, D, R, layout, dtype):
    m = 8 if D % 8 else 1  # heads a shard, so that its widths are multiples of 8 elements
    s = make(T, [3 * m, m], [m, 2 * m], D, dtype, seed=D + R)
    return s, proj_of(tp, T, s, dtype, D, rotary_dim=R, layout=layout, norm=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,R,layout", SHAPES)
def test_shapes(gpu_lib, D, R, layout, dtype):
    s, p = shape(gpu_lib, 37, D, R, layout, dtype)
    QK = p.qk_norm_rope_forward(s["QKV"], s["pos"])
    check_forward(s, QK, D, R, layout, dtype, norm=False, gains=False)
    dQKV, dgq, dgk = p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], dV_i=s["dV"])
    assert dgq is None and dgk is None
    check_backward(s, dQKV, None, None, D, R, layout, dtype, norm=False, gains=False)
    for x, dv, q, k in zip(dQKV, s["dV"], s["dq"], s["dkv"]):
        assert torch.equal(x[:, q + k:], dv)


@pytest.mark.parametrize("T", [1, 700, 9000])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
def test_backward_does_not_see_x(gpu_lib, bad, dtype, T):
    """Whatever stands in x, dx is that of dy."""
    s, p = shape(gpu_lib, T, 64, 32, "pairs", dtype)
    want = p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], dV_i=s["dV"])[0]
    spoiled = [torch.full_like(x, bad) for x in s["QKV"]]
    got = p.qk_norm_rope_backward(spoiled, s["dQK"], s["pos"], dV_i=s["dV"])[0]
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_backward_without_x(gpu_lib):
    """QKV need not be there; dense, in place, without dV, captured."""
    s, p = shape(gpu_lib, 301, 96, 96, "halves", "bf16")
    want = p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], dV_i=s["dV"])[0]
    got = p.qk_norm_rope_backward(None, s["dQK"], s["pos"], dV_i=s["dV"])[0]
    fused = [torch.cat([d, v], 1) for d, v in zip(s["dQK"], s["dV"])]
    kept = [x.clone() for x in fused]
    p.qk_norm_rope_backward(None, fused, s["pos"], out=fused)
    out = [torch.full_like(x, 7) for x in want]
    p.qk_norm_rope_backward(None, s["dQK"], s["pos"], out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = p.qk_norm_rope_backward(None, s["dQK"], s["pos"], dV_i=s["dV"])[0]
    graph.replay()
    for a, b, c, d, e, q, k in zip(want, got, fused, out, captured, s["dq"], s["dkv"]):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, e)
        assert torch.equal(a[:, :q + k], d[:, :q + k]) and (d[:, q + k:] == 7).all()
    assert all(torch.equal(x[:, q + k:], y[:, q + k:]) for x, y, q, k in zip(fused, kept, s["dq"], s["dkv"]))


def test_backward_turns_the_forward_pass_back(gpu_lib):
    """<rotate(x), dy> = <x, rotate back(dy)>, in fp32: both sums from the kernels' outputs, each off by 33 u (32, and
    the last rounding) of every term's magnitude |a||c| + |b||c|."""
    s, p = shape(gpu_lib, 400, 64, 32, "halves", "fp32")
    y = p.qk_norm_rope_forward(s["QKV"], s["pos"])
    dx = p.qk_norm_rope_backward(None, s["dQK"], s["pos"], dV_i=s["dV"])[0]
    for side in (q_of, k_of):
        x, c = heads(side(s, s["QKV"]), 64), heads(side(s, s["dQK"]), 64)
        bound = 33 * 2.0 ** -24 * ((ref.rotate_abs(x, 32, "halves") * np.abs(c)).sum()
                                   + (ref.rotate_abs(c, 32, "halves") * np.abs(x)).sum())
        assert abs((heads(side(s, y), 64) * c).sum() - (x * heads(side(s, dx), 64)).sum()) <= bound


@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_special_values_with_the_norm(gpu_lib, layout):
    """norm = 1, backward: a head of zeros and a huge one give the formula's gradient; a NaN and an infinity, in x or
    dy, spoil their own head and the gain's gradient of their kind, and nothing else."""
    s = make(40, [2], [2], 64, "fp32")
    x, dy = s["QKV"][0], s["dQK"][0]
    x[3, :64] = 0
    x[4, 64:128] *= 1e16
    p = proj_of(gpu_lib, 40, s, "fp32", 64, layout=layout)
    args = dict(positions=s["pos"], gq=s["gq"], gk=s["gk"], dV_i=s["dV"])
    clean, dgq, dgk = p.qk_norm_rope_backward(s["QKV"], s["dQK"], **args)
    check_backward(s, clean, dgq, dgk, 64, 64, layout, "fp32")
    x[6, 70] = float("nan")
    x[7, 5] = float("inf")
    dy[8, 3] = float("nan")
    got, dgq2, dgk2 = p.qk_norm_rope_backward(s["QKV"], s["dQK"], **args)
    a, b = np64(clean[0])[:, :256].reshape(40, 4, 64), np64(got[0])[:, :256].reshape(40, 4, 64)
    fine = np.ones((40, 4), bool)
    fine[6, 1] = fine[7, 0] = fine[8, 0] = False
    assert np.array_equal(a[fine], b[fine])
    assert np.isnan(b[6, 1]).all() and np.isnan(b[7, 0]).any() and np.isnan(b[8, 0]).all()
    assert dgq2.isnan().any() and torch.equal(dgk, dgk2)
    assert torch.equal(got[0][:, 256:], s["dV"][0])


@pytest.mark.parametrize("T", [1, 3, 640])
def test_many_shards_and_heads(gpu_lib, T):
    """The largest numbers of heads and shards; the same bits on another stream."""
    s = make(T, [64] * 16, [64] * 16, 32, "bf16")
    p = proj_of(gpu_lib, T, s, "bf16", 32, rotary_dim=16, layout="pairs", norm=False)
    check_forward(s, p.qk_norm_rope_forward(s["QKV"], s["pos"]), 32, 16, "pairs", "bf16", norm=False, gains=False)
    dQKV = p.qk_norm_rope_backward(None, s["dQK"], s["pos"], dV_i=s["dV"])[0]
    check_backward(s, dQKV, None, None, 32, 16, "pairs", "bf16", norm=False, gains=False)
    assert all(torch.equal(x[:, 4096:], v) for x, v in zip(dQKV, s["dV"]))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    again = p.qk_norm_rope_backward(None, s["dQK"], s["pos"], dV_i=s["dV"], stream=st)[0]
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(dQKV, again))


def test_no_tokens(gpu_lib):
    p = gpu_lib.ShardedAttentionProj(0, 64, [64], [64], "bf16")
    p.set_qk_norm_rope(64, norm=False)
    e = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device="cuda")
    assert p.qk_norm_rope_forward([e(192)])[0].shape == (0, 128)
    assert p.qk_norm_rope_backward(None, [e(128)], dV_i=[e(64)])[0][0].shape == (0, 192)


def test_gains_are_refused(gpu_lib):
    s, p = shape(gpu_lib, 20, 64, 64, "halves", "bf16")
    with pytest.raises(gpu_lib.TpmlpError):
        p.qk_norm_rope_forward(s["QKV"], s["pos"], s["gq"], s["gk"])
    with pytest.raises(gpu_lib.TpmlpError):
        p.qk_norm_rope_backward(None, s["dQK"], s["pos"], s["gq"], s["gk"], s["dV"])
    with pytest.raises(gpu_lib.TpmlpError):
        p.qk_norm_rope_backward(None, s["dQK"], s["pos"], dV_i=s["dV"], gain_grads=True)
    with pytest.raises(ValueError):  # with a norm x has to be there
        proj_of(gpu_lib, 20, s, "bf16", 64).qk_norm_rope_backward(None, s["dQK"], s["pos"], dV_i=s["dV"])
    with pytest.raises(ValueError):
        p.qk_norm_rope_forward(None, s["pos"])


def test_past_32_bits(gpu_lib):
    """Buffers of more than 2^32 bytes: the last tokens, against the same tokens alone."""
    T, n, last = 2_200_000, 1024, 70
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(5)
    big = lambda w: torch.randn(T, w, generator=gen, device="cuda", dtype=torch.bfloat16)
    x, dy, dv, pos = big(n), big(768), big(256), torch.arange(T, device="cuda")
    whole = gpu_lib.ShardedAttentionProj(T, 64, [512], [256])
    part = gpu_lib.ShardedAttentionProj(last, 64, [512], [256])
    for p in (whole, part):
        p.set_qk_norm_rope(128, rotary_dim=64, norm=False)
    cut = lambda t: t[-last:].contiguous()
    y = whole.qk_norm_rope_forward([x], pos)[0]
    assert torch.equal(y[-last:], part.qk_norm_rope_forward([cut(x)], cut(pos))[0])
    dx = whole.qk_norm_rope_backward(None, [dy], pos, dV_i=[dv])[0][0]
    assert torch.equal(dx[-last:], part.qk_norm_rope_backward(None, [cut(dy)], cut(pos), dV_i=[cut(dv)])[0][0])
