"""AdamW over many tensors, and the gradients' norm, against the definitions in 64 bits.

Bounds (u = 2^-24).  f: the norm 6 u (below) and a quotient, 8 u; x = f g: 9 u.  m: the betas as fp32 numbers, the
products and the sum: 4 u b1 |m| + 12 u (1 - b1) |f g|.  v: 4 u b2 v + 24 u (1 - b2) (f g)^2, all of one sign: below 24 u
of itself.  The root is off by 12 u and 2 u of its own, its correction 2 u, the sum with eps 2 u: the denominator by 18 u;
the quotient 4 u, lr / (1 - b1^t) 3 u: the update by dm lr_t / den + 26 u of itself; p by 3 u |p| and its last rounding.
A norm's squares are added 8 at a time (8 u of their sum), those sums without loss: 4 u of the root, the last rounding
and the workings of the pairs 2 u.

8-bit moments are a rising function of the moment for given random bits: what is kept has to lie between what the 64-bit
moment less and plus its bound would be kept as, with the group's scale either of those two groups'."""
import math

import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TD = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = [1, 7, 8, 255, 256, 257, 0, 2047, 4096, 4097, 5000, 100_003]
HYPER = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8)


def make(sizes, dtype, gdtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda n: torch.randn(n, generator=gen, device="cuda")
    p = [rnd(n).to(TD[dtype]) for n in sizes]

    def grads(k):
        gen.manual_seed(1000 * seed + k)
        gs = [1e-3 * rnd(n) * torch.exp(rnd(n)) for n in sizes]
        for g in gs:
            g[: g.numel() // 8] = 0
        return [g.to(TD[gdtype]) for g in gs]

    return p, grads


def within(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    assert ((got.double() - want).abs() <= bound).all(), (what, ((got.double() - want).abs() / bound).max().item())


def flat(xs):
    return torch.cat([x.reshape(-1) for x in xs])


class Copy:
    """The optimizer's state before a step, as 64-bit values."""

    def __init__(self, opt):
        self.p = [x.double() for x in (opt.master or opt.params)]
        if opt.bits == 32:
            self.m, self.v = [x.double() for x in opt.m], [x.double() for x in opt.v]
        else:
            self.m = [ref.values(b, n, False)[0] for b, n in zip(opt.m, opt.sizes)]
            self.v = [ref.values(b, n, True)[0] for b, n in zip(opt.v, opt.sizes)]


def check_step(opt, old, grads, norm, decays, grad_scale=1.0):
    t, (b1, b2), lr, eps = opt.steps, opt.betas, opt.lr, opt.eps
    f = grad_scale
    if norm is not None:
        exact = math.sqrt(sum((g.double() ** 2).sum().item() for g in grads))
        assert abs(norm.item() - exact) <= 6 * U * exact
        if exact * grad_scale > opt.max_norm:
            f = opt.max_norm / exact
    group0 = 0
    for k, n in enumerate(opt.sizes):
        if not n:
            continue
        p, m, v = ref.adamw(old.p[k], grads[k], old.m[k], old.v[k], t, lr, b1, b2, eps, decays[k], f)
        x = (grads[k].double() * f).abs()
        dm = 4 * U * b1 * old.m[k].abs() + 12 * U * (1 - b1) * x
        dv = 24 * U * v
        den = (v / (1 - b2 ** t)).sqrt() + eps
        rate = lr / (1 - b1 ** t)
        dp = dm * rate / den + 26 * U * rate * m.abs() / den + 3 * U * old.p[k].abs()
        if opt.master:
            within(opt.master[k], p, dp, f"master[{k}]")
            assert torch.equal(opt.params[k], opt.master[k].to(opt.tdtype))
        else:
            within(opt.params[k], p, dp + torch.finfo(opt.tdtype).eps / 2 * (p.abs() + dp), f"p[{k}]")
        if opt.bits == 32:
            within(opt.m[k], m, dm + 1e-44, f"m[{k}]")
            within(opt.v[k], v, dv + 1e-44, f"v[{k}]")
            continue
        groups = -(-n // ref.GROUP)
        r = ref.randoms(opt.seed, t, group0, groups, "cuda")
        group0 += groups
        for name, y, d, buf, second in (("m", m, dm, opt.m[k], False), ("v", v, dv, opt.v[k], True)):
            got, scale = ref.values(buf, n, second)
            pad = lambda z: torch.nn.functional.pad(z, (0, -n % ref.GROUP)).view(groups, ref.GROUP)
            y, d, got = pad(y), pad(d), pad(got)
            lo, hi = ((y.abs() + s * d).amax(1).clamp_min(0) for s in (-1, 1))
            e = scale.int() - 91
            zero = hi == 0
            assert torch.equal(scale == 0, zero), name
            ok = (e >= torch.where(zero, -91, ref.exponent(lo.clamp_min(1e-300)))) & \
                 (e <= torch.where(zero, -91, ref.exponent(hi.clamp_min(1e-300))))
            assert ok.all(), name
            least, most = (ref.rounded(y + s * d, e, r, second) for s in (-1, 1))
            assert ((got >= least) & (got <= most))[~zero].all(), (name, k)
            assert (got[zero] == 0).all()
            full = buf[:groups * ref.GROUP].view(-1)
            assert (full[n:] == 0).all()  # what fills up the last group


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("clip", [None, "below", "above"])
@pytest.mark.parametrize("dtype,gdtype,master", [("bf16", "bf16", False), ("bf16", "bf16", True), ("bf16", "fp32", True),
                                                 ("bf16", "fp32", False), ("fp32", "fp32", False),
                                                 ("fp32", "bf16", False)])
def test_steps(gpu_lib, dtype, gdtype, master, clip, bits):
    """The first steps from nothing, and one far on."""
    p, grads = make(SIZES, dtype, gdtype)
    decays = [0.1 if n > 300 else 0.0 for n in SIZES]
    size = math.sqrt(sum((g.double() ** 2).sum().item() for g in grads(0)))
    opt = gpu_lib.ShardedAdamW(p, **HYPER, weight_decay=decays, bits=bits, master=master, seed=(1 << 40) + 7,
                               max_norm={None: None, "below": 0.5 * size, "above": 20 * size}[clip])
    for k, lr in enumerate((1e-3, 2e-3, 5e-4, 1e-3)):
        if k == 3:
            opt.load_moments(opt.m, opt.v, steps=(1 << 33) + 5)
        old, g = Copy(opt), grads(k)
        norm = opt.step(g, lr=lr)
        check_step(opt, old, g, norm, decays)


@pytest.mark.parametrize("bits", [32, 8])
def test_grad_scale(gpu_lib, bits):
    p, grads = make(SIZES, "bf16", "bf16")
    size = math.sqrt(sum((g.double() ** 2).sum().item() for g in grads(0)))
    opt = gpu_lib.ShardedAdamW(p, **HYPER, bits=bits, max_norm=0.1 * size)
    for scale in (2.0 ** -4, 0.5):  # scaled below the limit, and above it
        old = Copy(opt)
        norm = opt.step(grads(0), grad_scale=scale)
        check_step(opt, old, grads(0), norm, [0.0] * len(SIZES), scale)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_holds(gpu_lib, bits):
    sizes = [1 + (37 * k) % 600 for k in range(900)]
    p, grads = make(sizes, "bf16", "bf16")
    opt = gpu_lib.ShardedAdamW(p, **HYPER, weight_decay=0.1, bits=bits, max_norm=1.0)
    for k in range(2):
        old, g = Copy(opt), grads(k)
        norm = opt.step(g)
        assert gpu_lib.tpmlp_last_launch_count() == 3
        check_step(opt, old, g, norm, [0.1] * len(sizes))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_skips_the_step(gpu_lib, bits, bad):
    p, grads = make(SIZES, "bf16", "bf16")
    opt = gpu_lib.ShardedAdamW(p, **HYPER, bits=bits, master=True, max_norm=1.0)
    opt.step(grads(0))
    before = [x.clone() for x in opt.params + opt.master + opt.m + opt.v]
    g = grads(1)
    g[9][4000] = bad
    norm = opt.step(g)
    assert not torch.isfinite(norm)
    assert all(torch.equal(a, b) for a, b in zip(before, opt.params + opt.master + opt.m + opt.v))
    old, g = Copy(opt), grads(2)
    norm = opt.step(g)  # the third step by number
    assert opt.steps == 3
    check_step(opt, old, g, norm, [0.0] * len(SIZES))


def test_a_bad_gradient_without_a_norm(gpu_lib):
    """It spoils its element, and, in 8 bits, its group's moments; nothing else."""
    for bits in (32, 8):
        p, grads = make([1000, 300], "fp32", "fp32")
        q = [x.clone() for x in p]
        a, b = (gpu_lib.ShardedAdamW(x, **HYPER, bits=bits) for x in (p, q))
        g = grads(0)
        a.step(g)
        g[0][700] = float("nan")
        b.step(g)
        assert torch.isnan(q[0][700])
        q[0][700] = p[0][700]
        assert all(torch.equal(x, y) for x, y in zip(p, q))
        for x, y in zip(sum(a.moments(), []), sum(b.moments(), [])):
            spoiled = torch.zeros_like(x, dtype=torch.bool)
            if x.numel() == 1000:
                spoiled[700 if bits == 32 else slice(512, 768)] = True
            assert torch.isnan(y[spoiled]).all() and torch.equal(x[~spoiled], y[~spoiled])
        b.step(grads(1))
        assert torch.isnan(b.moments()[0][0][700])


def test_moments_read_out(gpu_lib):
    p, grads = make(SIZES, "bf16", "bf16")
    opt = gpu_lib.ShardedAdamW(p, **HYPER, bits=8)
    for x in opt.moments():
        assert all((y == 0).all() for y in x)
    opt.step(grads(0))
    opt.step(grads(1))
    for got, bufs, second in zip(opt.moments(), (opt.m, opt.v), (False, True)):
        for x, b, n in zip(got, bufs, SIZES):
            assert x.dtype == torch.bfloat16 and torch.equal(x.double(), ref.values(b, n, second)[0])
    one = [torch.empty_like(x) for x in p]
    desc = gpu_lib.AdamWDesc(SIZES, "bf16", bits=8)
    gpu_lib.tpmlp_adamw8_unpack(desc, opt.m, None, one, None)
    assert all(torch.equal(a, b) for a, b in zip(one, opt.moments()[0]))
    gpu_lib.tpmlp_adamw8_unpack(desc, None, opt.v, None, one)
    assert all(torch.equal(a, b) for a, b in zip(one, opt.moments()[1]))


def test_every_code_comes_back(gpu_lib):
    """All 256 codes under scales from the smallest to the largest."""
    scales = torch.tensor([1, 2, 60, 91, 92, 150, 217], dtype=torch.uint8)
    n = 256 * len(scales)
    buf = torch.cat([torch.arange(256, dtype=torch.uint8).repeat(len(scales)), scales]).cuda()
    m, v = (torch.empty(n, dtype=torch.bfloat16, device="cuda") for _ in "mv")
    gpu_lib.tpmlp_adamw8_unpack(gpu_lib.AdamWDesc([n], "bf16", bits=8), [buf], [buf], [m], [v])
    assert torch.equal(m.double(), ref.values(buf, n, False)[0])
    assert torch.equal(v.double(), ref.values(buf, n, True)[0])


def test_stochastic_rounding_keeps_the_mean(gpu_lib):
    """100 steps without gradients: the second moment falls as 0.99^t in the mean, where rounding to the nearest code
    would keep it for ever.  A step's rounding is off by at most 1/16 of the value in the root of its mean square, 100 of
    them by 0.63; the mean of 2^16 elements by 0.0025: 1 % are four of those."""
    n = 1 << 16
    opt = gpu_lib.ShardedAdamW([torch.zeros(n, device="cuda")], lr=0.0, betas=(0.99, 0.99), bits=8, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(0)
    g = [1 + torch.rand(n, generator=gen, device="cuda")]
    opt.step(g)
    first = [x[0].double().mean().item() for x in opt.moments()]
    g[0].zero_()
    for _ in range(100):
        opt.step(g)
    for x, y in zip(first, opt.moments()):
        assert abs(y[0].double().mean().item() / (x * 0.99 ** 100) - 1) < 0.01


def test_the_second_moment_never_falls_to_zero(gpu_lib):
    """One large element in a group: the small ones' second moments stay above 0, and their steps bounded."""
    g = torch.full((256,), 1e-12, device="cuda")
    g[0] = 1e6
    p = torch.zeros(256, device="cuda")
    opt = gpu_lib.ShardedAdamW([p], lr=1e-3, eps=1e-30, bits=8)
    for _ in range(3):
        opt.step([g])
    m, v = opt.moments()
    assert (v[0] > 0).all() and (p.abs() <= 3.1e-3).all()


def test_the_seed_and_the_step_choose_the_rounding(gpu_lib):
    res = []
    for seed, steps in ((1, 0), (1, 0), (2, 0), (1 << 32, 0), (1, 1)):
        p, grads = make([5000], "bf16", "bf16")
        opt = gpu_lib.ShardedAdamW(p, **HYPER, bits=8, seed=seed)
        opt.load_moments(opt.m, opt.v, steps=steps)
        opt.step(grads(0))
        res.append(opt.m[0].clone())
    assert torch.equal(res[0], res[1])
    assert all(not torch.equal(res[0], x) for x in res[2:])


def test_nothing_is_written_past_the_end(gpu_lib):
    """Tensors of odd sizes that lie close to one another in one buffer."""
    for bits in (32, 8):
        buf = torch.full((4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        at = [(0, 13), (16, 1), (24, 250), (280, 257), (544, 1001)]
        p = [buf[a:a + n] for a, n in at]
        for x in p:
            x.fill_(1.0)
        inside = torch.zeros(4096, dtype=torch.bool, device="cuda")
        for a, n in at:
            inside[a:a + n] = True
        opt = gpu_lib.ShardedAdamW(p, **HYPER, bits=bits, max_norm=1.0)
        opt.step([torch.ones_like(x) for x in p])
        assert (buf[~inside] == 7.0).all() and (buf[inside] != 7.0).all()


def test_past_32_bit_offsets(gpu_lib):
    """One tensor of more than 2^32 elements: its last groups against the definition, the norm of all of it."""
    n = (1 << 32) + 1111
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-2000:] = torch.randn(2000, device="cuda").bfloat16()
    opt = gpu_lib.ShardedAdamW([p], **HYPER, bits=8, max_norm=1e9)
    norm = opt.step([g])
    exact = g[-2000:].double().norm().item()
    assert abs(norm.item() - exact) <= 6 * U * exact
    assert (p[:1 << 20] == 0).all() and (p[(1 << 32) - 4096:-2000] == 0).all()
    first = (n - 2000) // 256  # the groups from here on, as one tensor
    tail = n - first * 256
    cut = lambda b: torch.cat([b[first * 256: -(-n // 256) * 256], b[-tail // 256:]])
    want, m, v = ref.adamw(torch.zeros(tail, device="cuda"), g[-tail:], torch.zeros(tail, device="cuda"),
                           torch.zeros(tail, device="cuda"), 1, 1e-3, 0.9, 0.999, 1e-8, 0.0)
    assert ((p[-tail:].double() - want).abs() <= 2.0 ** -8 * 1.001 * want.abs()).all()
    r = ref.randoms(0, 1, first, -(-tail // 256), "cuda")
    pad = lambda z: torch.nn.functional.pad(z, (0, -tail % 256)).view(-1, 256)
    for y, buf, second in ((m, opt.m[0], False), (v, opt.v[0], True)):
        got, scale = ref.values(cut(buf), tail, second)
        e = scale.int() - 91
        least, most = (ref.rounded(pad(y * (1 + s * 24 * U)), e, r, second) for s in (-1, 1))
        lo, hi = torch.minimum(least, most), torch.maximum(least, most)
        assert ((pad(got) >= lo) & (pad(got) <= hi)).all()


def test_captured_steps_go_on_counting(gpu_lib):
    for bits in (32, 8):
        a, grads = make(SIZES, "bf16", "bf16")
        b, _ = make(SIZES, "bf16", "bf16")
        kw = dict(HYPER, bits=bits, master=True, max_norm=1.0, capturable=True)
        one, two = gpu_lib.ShardedAdamW(a, **kw), gpu_lib.ShardedAdamW(b, **kw)
        g = grads(0)
        for _ in range(4):
            one.step(g)
        two.step(g)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm = two.step(g)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert one.steps == two.steps == 4 and torch.isfinite(norm)
        for x, y in zip(one.params + one.master + one.m + one.v, two.params + two.master + two.m + two.v):
            assert torch.equal(x, y)
        old = Copy(two)
        two.lr_device.fill_(5e-4)
        two.lr = 5e-4  # what check_step goes by
        graph.replay()
        torch.cuda.synchronize()
        check_step(two, old, g, norm, [0.0] * len(SIZES))
    opt = gpu_lib.ShardedAdamW(a, **HYPER)
    x = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(ValueError, match="capturable"):
            opt.step(g)


def test_on_another_stream(gpu_lib):
    a, grads = make(SIZES, "bf16", "bf16")
    b, _ = make(SIZES, "bf16", "bf16")
    one, two = (gpu_lib.ShardedAdamW(x, **HYPER, bits=8, max_norm=1.0) for x in (a, b))
    g = grads(0)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    n1, n2 = one.step(g), two.step(g, stream=st)
    m1, m2 = one.moments(), two.moments(stream=st)
    torch.cuda.synchronize()
    assert torch.equal(n1, n2)
    assert all(torch.equal(x, y) for x, y in zip(a + m1[0] + m1[1], b + m2[0] + m2[1]))


@pytest.mark.parametrize("gdtype", ["bf16", "fp32"])
def test_norm(gpu_lib, gdtype):
    """Sizes from nothing to many CTAs, on a workspace that is used again."""
    ws = torch.zeros(gpu_lib.tpmlp_grad_norm_workspace_size(), dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(0)
    for sizes in ([], [0], [1], [0, 3, 0], SIZES, [1_000_003, 5], [30_000_001], [100] * 1001):
        g = [(torch.randn(n, generator=gen, device="cuda") * torch.exp(3 * torch.randn(n, generator=gen, device="cuda")))
             .to(TD[gdtype]) for n in sizes]
        desc = gpu_lib.AdamWDesc(sizes, gdtype)
        out = [torch.full((), -1.0, device="cuda") for _ in range(3)]
        for x in out:
            gpu_lib.tpmlp_grad_norm(desc, g, x, ws)
        exact = math.sqrt(sum((x.double() ** 2).sum().item() for x in g))
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
        assert abs(out[0].item() - exact) <= 6 * U * exact


def test_gradients_of_parameters(gpu_lib):
    """step() without a list takes .grad, as a program that trains with autograd calls it."""
    w = torch.randn(64, 32, device="cuda", requires_grad=True)
    b = torch.zeros(32, device="cuda", requires_grad=True)
    opt = gpu_lib.ShardedAdamW([w, b], lr=1e-2)
    with pytest.raises(ValueError, match="grad"):
        opt.step()
    x = torch.randn(16, 64, device="cuda")
    ((x @ w + b) ** 2).sum().backward()
    old = Copy(opt)
    opt.step()
    check_step(opt, old, [w.grad, b.grad], None, [0.0, 0.0])


def test_refusals_of_the_class(gpu_lib):
    tp = gpu_lib
    x = torch.zeros(64, 8, device="cuda", dtype=torch.bfloat16)
    for bad in ([], [x.half()], [x.cpu()], [x, x.float()], [x.t()]):
        with pytest.raises(ValueError):
            tp.ShardedAdamW(bad)
    for kw in (dict(bits=16), dict(weight_decay=[0.1, 0.2]), dict(max_norm=0.0), dict(max_norm=-1.0),
               dict(master=[x]), dict(master=[x.float(), x.float()])):
        with pytest.raises(ValueError):
            tp.ShardedAdamW([x], **kw)
    with pytest.raises(ValueError, match="fp32"):
        tp.ShardedAdamW([x.float()], master=True)
    opt = tp.ShardedAdamW([x])
    for bad in ([], [x, x], [x.half()], [x[:32]], [x.t().contiguous()], [x.cpu()]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(ValueError):
        opt.load_moments([x], [x])
    with pytest.raises(tp.TpmlpError) as e:
        opt.step([x])  # the gradient is the parameter
    assert e.value.status == 1
    y = torch.zeros(128, device="cuda")
    for twice in ([y, y], [y[:100], y[96:]]):
        with pytest.raises(tp.TpmlpError) as e:
            tp.ShardedAdamW(twice).step([torch.ones_like(t) for t in twice])
        assert e.value.status == 1
    assert (y == 0).all()
    for capturable in (False, True):
        opt = tp.ShardedAdamW([y], capturable=capturable)
        opt.step([torch.ones_like(y)])
        with pytest.raises(tp.TpmlpError):
            opt.step([y])
        assert opt.steps == 1  # a refused call is not a step
