"""The norm of the query and key heads with the position rotation, forward and backward, against its definition in
64 bits.

Bounds (u = 2^-24, before the last rounding to the storage type, which is off by at most eps / 2 of the value): the
sum of squares is at most 24 roundings deep (lane and tree), half of that in r, its reciprocal root 4 u, the two
products 2 u, sine and cosine 4 u and 3.2 u for the rounding of the angle to fp32, the combination 2 u: below 32 u of
|u_a| + |u_b|.  Backward: the same 32 u of r |s|, and 80 u of r |n| mean |s n| (each term 27 u, the mean's sum 24 u,
n 16 u, the rest below 13 u).  A gain's gradient adds T H terms of 27 u each, one after another at worst."""
import numpy as np
import pytest
import torch

import operators_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TD = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def half(dtype):
    return torch.finfo(TD[dtype]).eps / 2


def make(T, hq, hkv, D, dtype, seed=0, pos="packed"):
    """Random inputs: t shards of hq[i] query and hkv[i] key heads."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(TD[dtype]).cuda()
    dq, dkv = [D * h for h in hq], [D * h for h in hkv]
    s = {"QKV": [rnd(T, q + 2 * k) for q, k in zip(dq, dkv)], "dQK": [rnd(T, q + k) for q, k in zip(dq, dkv)],
         "dV": [rnd(T, k) for k in dkv], "gq": (1 + 0.2 * rnd(D)).to(TD[dtype]), "gk": (1 + 0.2 * rnd(D)).to(TD[dtype]),
         "dq": dq, "dkv": dkv}
    if pos == "packed":
        s["pos"] = (torch.randint(0, 5000, (T,), generator=gen)).cuda()
    elif pos == "far":
        s["pos"] = (torch.randint(-(1 << 24), 1 << 24, (T,), generator=gen)).cuda()
    else:
        s["pos"] = None
    return s


def proj_of(tp, T, s, dtype, D, **kw):
    p = tp.ShardedAttentionProj(T, 64, s["dq"], s["dkv"], dtype)
    p.set_qk_norm_rope(D, eps=EPS, **kw)
    return p


def np64(x):
    return x.detach().double().cpu().numpy()



def q_of(s, xs):
    return [(x, 0, w) for x, w in zip(xs, s["dq"])]


def k_of(s, xs):
    return [(x, o, w) for x, o, w in zip(xs, s["dq"], s["dkv"])]


def heads(parts, D):
    return np.concatenate([np64(x)[:, o:o + w].reshape(x.shape[0], w // D, D) for x, o, w in parts], 1)


def check(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} over, worst {np.max((np.abs(got - want) - bound)[bad])}"


def check_forward(s, QK, D, R, layout, dtype, norm=True, gains=True, freq=None):
    freq = ref.frequencies(R) if freq is None else freq
    pos = np.arange(QK[0].shape[0]) if s["pos"] is None else s["pos"].cpu().numpy()
    for what, side, g in (("q", q_of, "gq"), ("k", k_of, "gk")):
        x, y = heads(side(s, s["QKV"]), D), heads(side(s, QK), D)
        want, mag = ref.heads_forward(x, pos, freq, layout, np64(s[g]) if gains else 1.0, EPS, norm)
        check(y, want, half(dtype) * np.abs(want) + 32 * U * mag, what)


def check_backward(s, dQKV, dgq, dgk, D, R, layout, dtype, norm=True, gains=True, freq=None, dQK=None):
    freq = ref.frequencies(R) if freq is None else freq
    T = dQKV[0].shape[0]
    pos = np.arange(T) if s["pos"] is None else s["pos"].cpu().numpy()
    for what, side, g, dg in (("q", q_of, "gq", dgq), ("k", k_of, "gk", dgk)):
        x, dy = heads(side(s, s["QKV"]), D), heads(side(s, dQK or s["dQK"]), D)
        dx, dg64, mag, dgmag = ref.heads_backward(x, dy, pos, freq, layout, np64(s[g]) if gains else 1.0, EPS, norm)
        bound = half(dtype) * np.abs(dx) + U * (mag if norm else 32 * mag)
        check(heads(side(s, dQKV), D), dx, bound, "d" + what)
        if dg is not None:
            check(np64(dg), dg64, half(dtype) * np.abs(dg64) + (96 + T * x.shape[1]) * U * dgmag, "dg" + what)


# head sizes and rotated parts that take every vector width; sizes of the pages' attention shapes among them
SHAPES = [  # D, R, layout
    (128, 128, "halves"), (128, 128, "pairs"), (96, 96, "halves"), (96, 24, "halves"), (64, 32, "pairs"),
    (256, 256, "halves"), (256, 64, "pairs"), (80, 20, "halves"), (20, 10, "halves"), (20, 20, "pairs"),
    (8, 8, "halves"), (2, 2, "halves"), (2, 2, "pairs"), (64, 0, "halves"), (250, 126, "halves"), (254, 254, "pairs"),
    (252, 252, "halves"), (252, 100, "pairs"), (244, 20, "halves"), (132, 132, "halves"), (4, 4, "pairs"),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,R,layout", SHAPES)
def test_shapes(gpu_lib, D, R, layout, dtype):
    """Two unequal shards; heads per shard such that the widths are multiples of 16 bytes."""
    m = 8 if D % 8 else 1  # heads a shard, so that its widths are multiples of 8 elements
    s = make(37, [3 * m, m], [m, 2 * m], D, dtype, seed=D + R)
    p = proj_of(gpu_lib, 37, s, dtype, D, rotary_dim=R, layout=layout)
    QK = p.qk_norm_rope_forward(s["QKV"], positions=s["pos"], gq=s["gq"], gk=s["gk"])
    check_forward(s, QK, D, R, layout, dtype)
    dQKV, dgq, dgk = p.qk_norm_rope_backward(s["QKV"], s["dQK"], positions=s["pos"], gq=s["gq"], gk=s["gk"],
                                             dV_i=s["dV"])
    check_backward(s, dQKV, dgq, dgk, D, R, layout, dtype)
    for x, dv, q, k in zip(dQKV, s["dV"], s["dq"], s["dkv"]):
        assert torch.equal(x[:, q + k:], dv)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 31, 333, 2500])
def test_lengths(gpu_lib, T, dtype):
    """One token (its heads split over warps) to more tokens than the GPU has warps; 3 shards, grouped keys."""
    s = make(T, [16, 4, 1], [1, 4, 1], 64, dtype, seed=T)
    p = proj_of(gpu_lib, T, s, dtype, 64)
    check_forward(s, p.qk_norm_rope_forward(s["QKV"], s["pos"], s["gq"], s["gk"]), 64, 64, "halves", dtype)
    check_backward(s, *p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], s["gq"], s["gk"], s["dV"]), 64, 64,
                   "halves", dtype)


def test_many_shards_and_heads_of_one_token(gpu_lib):
    s = make(1, [64] * 16, [64] * 16, 32, "bf16")
    p = proj_of(gpu_lib, 1, s, "bf16", 32)
    check_forward(s, p.qk_norm_rope_forward(s["QKV"], s["pos"], s["gq"], s["gk"]), 32, 32, "halves", "bf16")
    check_backward(s, *p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], s["gq"], s["gk"], s["dV"]), 32, 32,
                   "halves", "bf16")


@pytest.mark.parametrize("pos", ["far", None])
def test_positions(gpu_lib, pos):
    """Positions of millions, negative ones, and none given.  fp32, so that the angle's error shows: 2^24 radians
    in 64 bits are off by 2^24 2^-53 2 at most, below u / 32."""
    s = make(200, [2], [2], 64, "fp32", pos=pos)
    p = proj_of(gpu_lib, 200, s, "fp32", 64)
    check_forward(s, p.qk_norm_rope_forward(s["QKV"], s["pos"], s["gq"], s["gk"]), 64, 64, "halves", "fp32")


def test_given_frequencies(gpu_lib):
    """inv_freq instead of the base: negative, zero and more than a turn per position."""
    s = make(65, [2], [1], 16, "fp32")
    freq = np.array([0.5, -0.25, 0.0, 7.0, -1e-18, 1.0, 6.283185307179586, 1e-5])
    p = proj_of(gpu_lib, 65, s, "fp32", 16, inv_freq=list(freq))
    check_forward(s, p.qk_norm_rope_forward(s["QKV"], s["pos"], s["gq"], s["gk"]), 16, 16, "halves", "fp32", freq=freq)


@pytest.mark.parametrize("norm", [True, False])
def test_without_gains_or_norm(gpu_lib, norm):
    s = make(50, [3], [2], 64, "bf16")
    p = proj_of(gpu_lib, 50, s, "bf16", 64, norm=norm)
    QK = p.qk_norm_rope_forward(s["QKV"], s["pos"])
    check_forward(s, QK, 64, 64, "halves", "bf16", norm=norm, gains=False)
    dQKV, dgq, dgk = p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], dV_i=s["dV"], gain_grads=norm)
    check_backward(s, dQKV, dgq, dgk, 64, 64, "halves", "bf16", norm=norm, gains=False)


def test_in_place(gpu_lib):
    """Forward over QKV itself and backward over dQKV itself: the bits of the other form, the value columns kept."""
    s = make(301, [4, 2], [2, 1], 96, "bf16")
    p = proj_of(gpu_lib, 301, s, "bf16", 96)
    args = dict(positions=s["pos"], gq=s["gq"], gk=s["gk"])
    QK = p.qk_norm_rope_forward(s["QKV"], **args)
    own = [x.clone() for x in s["QKV"]]
    out = p.qk_norm_rope_forward(own, out=own, **args)
    dQKV, dgq, dgk = p.qk_norm_rope_backward(s["QKV"], s["dQK"], dV_i=s["dV"], **args)
    fused = [torch.cat([d, v], 1) for d, v in zip(s["dQK"], s["dV"])]
    got, dgq2, dgk2 = p.qk_norm_rope_backward(s["QKV"], fused, out=fused, **args)
    for i, (q, k) in enumerate(zip(s["dq"], s["dkv"])):
        assert out[i] is own[i] and torch.equal(own[i][:, :q + k], QK[i])
        assert torch.equal(own[i][:, q + k:], s["QKV"][i][:, q + k:])
        assert torch.equal(got[i], dQKV[i])
    assert torch.equal(dgq, dgq2) and torch.equal(dgk, dgk2)


def test_special_values(gpu_lib):
    """A head of zeros, tiny and huge heads, and a NaN and an infinity that spoil their own head only."""
    s = make(40, [2], [2], 64, "fp32")
    x = s["QKV"][0]
    x[3, :64] = 0
    x[4, :64] = 1e-30
    x[5, :64] *= 1e16
    x[6, 70] = float("nan")
    x[7, 5] = float("inf")
    p = proj_of(gpu_lib, 40, s, "fp32", 64)
    y = np64(p.qk_norm_rope_forward(s["QKV"], s["pos"], s["gq"], s["gk"])[0]).reshape(40, 4, 64)
    xs = np64(x)[:, :256].reshape(40, 4, 64)
    g = np.stack([np64(s["gq"])] * 2 + [np64(s["gk"])] * 2)[None]
    with np.errstate(invalid="ignore"):
        want, mag = ref.heads_forward(xs, s["pos"].cpu().numpy(), ref.frequencies(64), "halves", g, EPS)
    fine = np.ones((40, 4), bool)
    fine[6, 1] = fine[7, 0] = False
    check(y[fine], want[fine], 2.0 ** -24 * np.abs(want[fine]) + 32 * U * mag[fine] + 1e-37, "special")
    assert np.isnan(y[6, 1]).all() and np.isnan(y[7, 0]).any()
    assert (y[3, 0] == 0).all()


def test_same_bits_every_time_and_on_other_streams(gpu_lib):
    s = make(1000, [8, 4], [2, 2], 64, "bf16")
    p = proj_of(gpu_lib, 1000, s, "bf16", 64)
    args = dict(positions=s["pos"], gq=s["gq"], gk=s["gk"])
    first = p.qk_norm_rope_backward(s["QKV"], s["dQK"], dV_i=s["dV"], **args)
    y = p.qk_norm_rope_forward(s["QKV"], **args)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    again = p.qk_norm_rope_backward(s["QKV"], s["dQK"], dV_i=s["dV"], stream=st, **args)
    y2 = p.qk_norm_rope_forward(s["QKV"], stream=st.cuda_stream, **args)
    st.synchronize()
    for a, b in zip(first[0] + [first[1], first[2]] + y, again[0] + [again[1], again[2]] + y2):
        assert torch.equal(a, b)


def test_captured_and_replayed(gpu_lib):
    s = make(500, [4], [2], 128, "bf16")
    p = proj_of(gpu_lib, 500, s, "bf16", 128)
    args = dict(positions=s["pos"], gq=s["gq"], gk=s["gk"])
    p.qk_norm_rope_backward(s["QKV"], s["dQK"], dV_i=s["dV"], **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        QK = p.qk_norm_rope_forward(s["QKV"], **args)
        dQKV, dgq, dgk = p.qk_norm_rope_backward(s["QKV"], s["dQK"], dV_i=s["dV"], **args)
    new = make(500, [4], [2], 128, "bf16", seed=9)
    for k in ("QKV", "dQK", "dV"):
        s[k][0].copy_(new[k][0])
    s["pos"].copy_(new["pos"])
    graph.replay()
    torch.cuda.synchronize()
    check_forward(s, QK, 128, 128, "halves", "bf16")
    check_backward(s, dQKV, dgq, dgk, 128, 128, "halves", "bf16")


def test_gradient_against_differences(gpu_lib):
    """The kernels' backward pass against central differences of the kernels' forward pass, in fp32, along random
    directions of x and of the gains.  L = sum(y c); h = 2^-6: the differences' own error is h^2 / 6 of the third
    derivative (below 2^-12 of the scale here) and 2 u of L's terms over h."""
    s = make(60, [2], [1], 32, "fp32")
    p = proj_of(gpu_lib, 60, s, "fp32", 32)
    c = s["dQK"][0].double()
    dQKV, dgq, dgk = p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], s["gq"], s["gk"], s["dV"])
    gen = torch.Generator().manual_seed(3)
    rnd = lambda x: torch.randn(x.shape, generator=gen).cuda()
    vx, vq, vk = rnd(s["QKV"][0]), rnd(s["gq"]), rnd(s["gk"])
    vx[:, 96:] = 0

    def L(h):
        y = p.qk_norm_rope_forward([s["QKV"][0] + h * vx], s["pos"], s["gq"] + h * vq, s["gk"] + h * vk)[0]
        return (y.double() * c).sum().item()

    h = 2.0 ** -6
    diff = (L(h) - L(-h)) / (2 * h)
    want = (dQKV[0].double() * vx.double()).sum() + (dgq.double() * vq.double()).sum() + (dgk.double() * vk.double()).sum()
    scale = (dQKV[0].double() * vx.double()).norm() + (dgq * vq).norm() + (dgk * vk).norm()
    assert abs(diff - want.item()) <= 2e-2 * scale.item()


def test_empty(gpu_lib):
    p = gpu_lib.ShardedAttentionProj(0, 64, [64], [64], "bf16")
    p.set_qk_norm_rope(64)
    e = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    assert p.qk_norm_rope_forward([e(192)], gq=g, gk=g)[0].shape == (0, 128)
    dQKV, dgq, dgk = p.qk_norm_rope_backward([e(192)], [e(128)], gq=g, gk=g, dV_i=[e(64)])
    assert dQKV[0].shape == (0, 192) and not dgq.any() and not dgk.any()


def test_two_threads_on_two_streams(gpu_lib):
    """Two host threads, each with its plan, workspace and stream, at the same time: the bits of one after the
    other."""
    import threading
    jobs = []
    for seed, (T, hq, hkv, D, layout) in enumerate([(700, [4, 2], [2, 1], 96, "halves"), (900, [8], [2], 64, "pairs")]):
        s = make(T, hq, hkv, D, "bf16", seed=seed)
        p = proj_of(gpu_lib, T, s, "bf16", D, layout=layout)
        call = lambda p=p, s=s, **kw: p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], s["gq"], s["gk"], s["dV"],
                                                              **kw)
        jobs.append((call, call()))
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            st = torch.cuda.Stream()
            for _ in range(20):
                got[i].append(jobs[i][0](stream=st))
            st.synchronize()
        except Exception as e:  # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for (_, (dQKV, dgq, dgk)), runs in zip(jobs, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(dQKV + [dgq, dgk], r[0] + [r[1], r[2]]))


def test_python_refusals(gpu_lib):
    """Wrong shapes, types, strides and devices are refused before any launch."""
    s = make(20, [2], [2], 32, "bf16")
    p = proj_of(gpu_lib, 20, s, "bf16", 32)
    bad = [dict(QKV_i=[s["QKV"][0][:10]]), dict(QKV_i=[s["QKV"][0].float()]), dict(QKV_i=[s["QKV"][0].cpu()]),
           dict(QKV_i=[s["QKV"][0].t().contiguous().t()]), dict(QKV_i=s["QKV"] * 2),
           dict(positions=s["pos"].int()), dict(positions=s["pos"][:5]), dict(positions=s["pos"].cpu()),
           dict(gq=s["gq"][:16]), dict(gk=s["gk"].float()), dict(out=[torch.empty_like(s["QKV"][0])]), dict(out=[])]
    for kw in bad:
        with pytest.raises(ValueError):
            p.qk_norm_rope_forward(**{**dict(QKV_i=s["QKV"], positions=s["pos"], gq=s["gq"], gk=s["gk"]), **kw})
    with pytest.raises(ValueError):  # nothing says where dV comes from
        p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], s["gq"], s["gk"])
    with pytest.raises(ValueError):
        gpu_lib.ShardedAttentionProj(20, 64, [64], [64]).qk_norm_rope_forward(s["QKV"])
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    f = proj_of(gpu_lib, 20, make(20, [2], [2], 32, "fp32"), "fp32", 32)
    with pytest.raises(ValueError):  # a workspace from before the norm was described
        gpu_lib.tpmlp_attn_qk_norm_rope_backward(f.plan, [1 << 20], None, None, None, [1 << 22], None, [1 << 24],
                                                 1 << 26, None, small)


def test_past_32_bits(gpu_lib):
    """Buffers of more than 2^32 bytes: the last tokens, against the same tokens alone."""
    T, n, last = 2_200_000, 1024, 70
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(5)
    big = lambda w: torch.randn(T, w, generator=gen, device="cuda", dtype=torch.bfloat16)
    x, dy, dv = big(n), big(768), big(256)
    pos = torch.arange(T, device="cuda")
    g = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    whole = gpu_lib.ShardedAttentionProj(T, 64, [512], [256])
    part = gpu_lib.ShardedAttentionProj(last, 64, [512], [256])
    for p in (whole, part):
        p.set_qk_norm_rope(128)
    cut = lambda t: t[-last:].contiguous()
    y = whole.qk_norm_rope_forward([x], pos, g, g)[0]
    assert torch.equal(y[-last:], part.qk_norm_rope_forward([cut(x)], cut(pos), g, g)[0])
    dx = whole.qk_norm_rope_backward([x], [dy], pos, g, g, [dv])[0][0]
    want = part.qk_norm_rope_backward([cut(x)], [cut(dy)], cut(pos), g, g, [cut(dv)])[0][0]
    assert torch.equal(dx[-last:], want)
