"""The tokens' norm, forward and backward, against its definition in 64 bits.

Bounds (u = 2^-24; h = eps / 2 of the storage type for the last rounding).  A sum over a token is 32 elements one after
another, 5 shuffles and up to 16 warps: at most 53 roundings deep.  Forward: the mean is off by delta = 56 u mean|s|
(its division by d among them).  The sum of squares of s - mu is off by 60 u relative (53, the squares 2, the difference
2, the product with 1 / d and eps 3) and by delta^2 for the mean (a shift of the mean adds its square), r by half of that
and 6 u (the reciprocal root 4, one product 2): rho.  y by |g| r delta for the mean, |s - mu| r |g| (rho + 4 u), 2 u |b|.
Backward, from the statistics as they are: n 2 u, w 1 u, their products 1 u; mean(w) 56 u mean|w|, mean(w n) 60 u
mean|w n|; three roundings of the combination: in all r (6 u |w| + 62 u mean|w| + 68 u |n| mean|w n|) + 2 u |dsum|.  A
gradient of gain or bias adds T terms of 3 u each, one after another at worst, and 80 partial sums."""
import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TD = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def half(dtype):
    return torch.finfo(TD[dtype]).eps / 2


def make(T, d, dtype, seed=0, shift=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    to = lambda x: x.to(TD[dtype])
    return {"x": to(rnd(T, d) * torch.exp(0.5 * rnd(d)) + shift), "r": to(rnd(T, d)), "dy": to(rnd(T, d)),
            "ds": to(rnd(T, d)), "g": to(1 + 0.2 * rnd(d)), "b": to(0.2 * rnd(d))}


def within(got, want, bound):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    worst = (err / bound.clamp_min(1e-300)).max().item() if err.numel() else 0.0
    assert (err <= bound).all(), worst


def check_forward(y, stats, s, g, b, kind, dtype):
    want, mu, r = ref.norm_forward(s, g, b, kind, EPS)
    s64 = s.double()
    delta = 56 * U * s64.abs().mean(1) if kind == "layer" else torch.zeros_like(mu)
    rho = 36 * U + delta ** 2 * r ** 2 / 2
    within(stats[:, 0], mu, delta + U * mu.abs())
    within(stats[:, 1], r, rho * r)
    ga = torch.ones_like(s64[0]) if g is None else g.double().abs()
    c = (s64 - mu[:, None]).abs()
    bound = ga * (r * delta)[:, None] + c * r[:, None] * ga * (rho + 4 * U)[:, None] + half(dtype) * 1.001 * want.abs()
    if b is not None:
        bound = bound + 2 * U * b.double().abs()
    within(y, want, bound)


def check_backward(got, s, stats, dy, ds, g, kind, dtype):
    dx, dg, db = got
    want, wg, wb = ref.norm_backward(s, stats[:, 0], stats[:, 1], dy, ds, g, kind)
    n = ((s.double() - stats[:, :1].double()) * stats[:, 1:].double()).abs()
    w = dy.double().abs() * (1.0 if g is None else g.double().abs())
    bound = stats[:, 1:].double() * (6 * U * w + 62 * U * w.mean(1, keepdim=True) +
                                     68 * U * n * (w * n).mean(1, keepdim=True)) + half(dtype) * 1.001 * want.abs()
    if ds is not None:
        bound = bound + 2 * U * ds.double().abs()
    within(dx, want, bound)
    T = s.shape[0]
    if dg is not None:
        within(dg, wg, (T + 83) * U * (dy.double().abs() * n).sum(0) + half(dtype) * 1.001 * wg.abs())
    if db is not None:
        within(db, wb, (T + 83) * U * dy.double().abs().sum(0) + half(dtype) * 1.001 * wb.abs())


# widths of each team size, at its ends and between; rows from one to more than the launch has teams
SHAPES = [(1, 8), (1, 4096), (2, 264), (3, 512), (5, 520), (7, 1024), (9, 1032), (33, 2048), (3, 2056), (161, 4096),
          (5, 4104), (2, 8192), (4, 8200), (153, 16384), (2500, 256), (5000, 40), (1300, 768)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_and_backward(gpu_lib, T, d, kind, dtype):
    a = make(T, d, dtype, seed=T + d)
    norm = gpu_lib.TokenNorm(T, d, kind, dtype, eps=EPS)
    bias = a["b"] if kind == "layer" else None
    y, stats, s = norm.forward(a["x"], a["g"], bias, residual=a["r"])
    exact = a["x"].double() + a["r"].double()
    within(s, exact, (half(dtype) * 1.001 + U) * exact.abs())
    check_forward(y, stats, s, a["g"], bias, kind, dtype)
    check_backward(norm.backward(s, stats, a["dy"], a["g"], dsum=a["ds"], bias_grad=kind == "layer"), s, stats,
                   a["dy"], a["ds"], a["g"], kind, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_without_the_options(gpu_lib, kind, dtype):
    """No residual, no gain, no bias, no dsum, and each gradient by itself."""
    T, d = 37, 1544
    a = make(T, d, dtype)
    norm = gpu_lib.TokenNorm(T, d, kind, dtype, eps=EPS)
    y, stats, s = norm.forward(a["x"])
    assert s is a["x"]
    check_forward(y, stats, s, None, None, kind, dtype)
    got = norm.backward(s, stats, a["dy"])
    assert got[1] is None and got[2] is None
    check_backward(got, s, stats, a["dy"], None, None, kind, dtype)
    both = norm.backward(s, stats, a["dy"], gain_grad=True, bias_grad=True)
    for gain, bias in ((True, False), (False, True)):
        one = norm.backward(s, stats, a["dy"], gain_grad=gain, bias_grad=bias)
        assert torch.equal(one[0], both[0])
        assert (one[1] is None) == (not gain) and (one[2] is None) == (not bias)
        assert torch.equal(one[1] if gain else one[2], both[1] if gain else both[2])
    y2, stats2, _ = norm.forward(a["x"], None, a["b"])
    check_forward(y2, stats2, s, None, a["b"], kind, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_mean_far_from_zero(gpu_lib, dtype):
    a = make(65, 4096, dtype, shift=3000.0)
    norm = gpu_lib.TokenNorm(65, 4096, "layer", dtype, eps=EPS)
    y, stats, s = norm.forward(a["x"], a["g"], a["b"])
    check_forward(y, stats, s, a["g"], a["b"], "layer", dtype)
    check_backward(norm.backward(s, stats, a["dy"], a["g"], bias_grad=True), s, stats, a["dy"], None, a["g"], "layer",
                   dtype)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_rows_of_one_value(gpu_lib, kind):
    """No spread at all: n is 0 (layer), eps alone keeps r finite."""
    norm = gpu_lib.TokenNorm(3, 512, kind, "fp32", eps=EPS)
    x = torch.zeros(3, 512, device="cuda")
    x[1] = 0.5  # a sum of 512 halves and its mean are exact
    y, stats, _ = norm.forward(x)
    check_forward(y, stats, x, None, None, kind, "fp32")
    if kind == "layer":
        assert (y == 0).all()
    dx = norm.backward(x, stats, torch.ones_like(x))[0]
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("d", [64, 4096])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_spoils_itself_only(gpu_lib, d, bad):
    T = 400
    a = make(T, d, "bf16")
    norm = gpu_lib.TokenNorm(T, d, "layer", "bf16", eps=EPS)
    want = norm.forward(a["x"], a["g"], a["b"], residual=a["r"])
    dwant = norm.backward(want[2], want[1], a["dy"], a["g"], dsum=a["ds"])[0]
    x = a["x"].clone()
    x[7, d // 2] = bad
    got = norm.forward(x, a["g"], a["b"], residual=a["r"])
    dgot = norm.backward(got[2], got[1], a["dy"], a["g"], dsum=a["ds"])[0]
    keep = torch.arange(T, device="cuda") != 7
    for u, v in zip(want + (dwant,), got + (dgot,)):
        assert torch.equal(u[keep], v[keep])
    assert torch.isnan(got[0][7]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_apart(gpu_lib, dtype):
    """Column slices in and out, of one buffer too; what lies between the rows stays as it was."""
    T, d, wide = 77, 264, 600
    a = make(T, d, dtype)
    norm = gpu_lib.TokenNorm(T, d, "layer", dtype, eps=EPS)
    y, stats, s = norm.forward(a["x"], a["g"], a["b"], residual=a["r"])
    dx, dg, db = norm.backward(s, stats, a["dy"], a["g"], dsum=a["ds"], bias_grad=True)

    def spread(x, at):
        big = torch.full((T, wide), 7.0, dtype=x.dtype, device="cuda")
        big[:, at:at + d] = x
        return big, big[:, at:at + d]

    (_, xs), (_, rs), (_, dys), (_, dss) = (spread(a[k], o) for k, o in (("x", 8), ("r", 0), ("dy", 16), ("ds", 24)))
    (yb, ys), (sb, ss) = spread(torch.zeros_like(y), 32), spread(torch.zeros_like(s), 40)
    y2, stats2, s2 = norm.forward(xs, a["g"], a["b"], residual=rs, out=(ys, ss))
    assert torch.equal(y2, y) and torch.equal(s2, s) and torch.equal(stats2, stats)
    db_, dxs = spread(torch.zeros_like(dx), 48)
    got = norm.backward(ss, stats, dys, a["g"], dsum=dss, out=dxs, bias_grad=True)
    assert torch.equal(dxs, dx) and torch.equal(got[1], dg) and torch.equal(got[2], db)
    for big, at in ((yb, 32), (sb, 40), (db_, 48)):
        assert (big[:, :at] == 7.0).all() and (big[:, at + d:] == 7.0).all()
    big = torch.zeros(T, 2 * d + 16, dtype=TD[dtype], device="cuda")  # x and y side by side in one buffer
    big[:, :d] = a["x"]
    out = norm.forward(big[:, :d], a["g"], a["b"], out=(big[:, d + 8:2 * d + 8], None))
    assert torch.equal(out[0], norm.forward(a["x"], a["g"], a["b"])[0]) and torch.equal(big[:, :d], a["x"])


@pytest.mark.parametrize("T,d", [(50, 264), (700, 4096)])
def test_in_place(gpu_lib, T, d):
    a = make(T, d, "bf16")
    norm = gpu_lib.TokenNorm(T, d, "layer", "bf16", eps=EPS)
    y, stats, s = norm.forward(a["x"], a["g"], a["b"], residual=a["r"])
    dx = norm.backward(s, stats, a["dy"], a["g"], dsum=a["ds"])[0]
    plain = norm.forward(a["x"], a["g"], a["b"])[0]
    for s_is, y_is in (("x", None), ("r", None), (None, "x"), (None, "r"), ("x", "r"), ("r", "x")):
        c = {k: v.clone() for k, v in a.items()}
        out = (c[y_is] if y_is else torch.empty_like(y), c[s_is] if s_is else torch.empty_like(s))
        got = norm.forward(c["x"], c["g"], c["b"], residual=c["r"], out=out)
        assert torch.equal(got[0], y) and torch.equal(got[2], s) and torch.equal(got[1], stats)
    c = a["x"].clone()
    assert torch.equal(norm.forward(c, a["g"], a["b"], out=(c, None))[0], plain)
    for k in ("dy", "ds", "s"):
        c = {"dy": a["dy"].clone(), "ds": a["ds"].clone(), "s": s.clone()}
        assert torch.equal(norm.backward(c["s"], stats, c["dy"], a["g"], dsum=c["ds"], out=c[k])[0], dx)


def test_no_tokens(gpu_lib):
    norm = gpu_lib.TokenNorm(0, 64, "layer", "bf16")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, stats, s = norm.forward(x, g, g, residual=x)
    dx, dg, db = norm.backward(s, stats, x, g, bias_grad=True)
    assert y.shape == dx.shape == (0, 64) and (dg == 0).all() and (db == 0).all()


def test_past_32_bit_offsets(gpu_lib):
    """Rows 16384 elements apart, the last ones beyond 2^32 bytes and 2^31 elements."""
    T, d, ld = 140_000, 64, 16384
    a = make(T, d, "bf16")
    norm = gpu_lib.TokenNorm(T, d, "layer", "bf16", eps=EPS)
    y, stats, s = norm.forward(a["x"], a["g"], a["b"])
    dx, dg, _ = norm.backward(s, stats, a["dy"], a["g"])
    big = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")
    x, y2, dy, dx2 = (big[:, k * 64:(k + 1) * 64] for k in range(4))
    x.copy_(a["x"])
    dy.copy_(a["dy"])
    got = norm.forward(x, a["g"], a["b"], out=(y2, None))
    assert torch.equal(y2, y) and torch.equal(got[1], stats)
    got = norm.backward(x, stats, dy, a["g"], out=dx2)
    assert torch.equal(dx2, dx) and torch.equal(got[1], dg)


def test_same_result_on_every_run_on_another_stream_and_in_a_graph(gpu_lib):
    T, d = 1000, 2048
    a = make(T, d, "bf16")
    norm = gpu_lib.TokenNorm(T, d, "layer", "bf16", eps=EPS)

    def both(**kw):
        y, stats, s = norm.forward(a["x"], a["g"], a["b"], residual=a["r"], **kw)
        return (y, stats, s) + norm.backward(s, stats, a["dy"], a["g"], dsum=a["ds"], bias_grad=True, **kw)

    want = both()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = both(stream=st)
    st.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for v in got:
        v.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("residual", [True, False])
def test_autograd(gpu_lib, kind, residual):
    """The autograd function's gradients against torch's own of the definition in 64 bits, where y and the sum are both
    used; 1e-5 of the largest entry: the bounds above sum to less for 48 tokens of 256 elements."""
    T, d = 48, 256
    a = {k: v.requires_grad_() for k, v in make(T, d, "fp32").items()}
    norm = gpu_lib.TokenNorm(T, d, kind, "fp32", eps=EPS)
    bias = a["b"] if kind == "layer" else None
    args = (norm, a["x"], a["g"], bias) + ((a["r"],) if residual else ())
    leaves = [a["x"], a["g"]] + ([a["b"]] if bias is not None else []) + ([a["r"]] if residual else [])
    out = gpu_lib.TPMLPNormFunction.apply(*args)
    y, s = out if residual else (out, None)
    loss = (y * a["dy"].detach()).sum() + ((s * a["ds"].detach()).sum() if residual else 0)
    got = torch.autograd.grad(loss, leaves)
    c = {k: v.detach().double().requires_grad_() for k, v in a.items()}
    s64 = c["x"] + c["r"] if residual else c["x"]
    y64 = ref.norm_forward(s64, c["g"], c["b"] if bias is not None else None, kind, EPS)[0]
    loss = (y64 * c["dy"].detach()).sum() + ((s64 * c["ds"].detach()).sum() if residual else 0)
    names = ["x", "g"] + (["b"] if bias is not None else []) + (["r"] if residual else [])
    for u, v in zip(got, torch.autograd.grad(loss, [c[k] for k in names])):
        assert (u.double() - v).abs().max() <= 1e-5 * v.abs().max()
    if residual:  # only one of the two outputs used
        for k in (0, 1):
            out = gpu_lib.TPMLPNormFunction.apply(*args)
            got = torch.autograd.grad((out[k] * a["dy"].detach()).sum(), [a["x"], a["r"]])
            s64 = c["x"] + c["r"]
            o64 = s64 if k else ref.norm_forward(s64, c["g"], c["b"] if bias is not None else None, kind, EPS)[0]
            v = torch.autograd.grad((o64 * c["dy"].detach()).sum(), c["x"])[0]
            assert all((u.double() - v).abs().max() <= 1e-5 * v.abs().max() for u in got)


def test_autograd_of_other_layouts(gpu_lib):
    """A frozen gain, gradients that arrive expanded or transposed, rows at a distance that is no whole number of 16
    bytes."""
    T, d = 24, 64
    a = make(T, d, "fp32")
    norm = gpu_lib.TokenNorm(T, d, "layer", "fp32", eps=EPS)
    want = gpu_lib.TPMLPNormFunction.apply(norm, a["x"], a["g"], a["b"])
    wide = torch.zeros(T, d + 3, device="cuda")
    wide[:, :d] = a["x"]
    x = wide[:, :d].requires_grad_()
    y = gpu_lib.TPMLPNormFunction.apply(norm, x, a["g"], a["b"])
    assert torch.equal(y, want)
    for dy in (torch.ones((), device="cuda").expand(T, d), a["dy"].t().contiguous().t(), a["dy"]):
        got = torch.autograd.grad(y, x, dy, retain_graph=True)[0]
        s, stats = norm.forward(a["x"], a["g"], a["b"])[2:0:-1]
        assert torch.equal(got, norm.backward(s, stats, dy.contiguous(), a["g"])[0])
        assert gpu_lib.tpmlp_last_launch_count() == 2
    y.sum().backward()
    assert a["g"].grad is None and x.grad is not None
