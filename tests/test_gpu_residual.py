"""The row-parallel products with the residual stream in their epilogue, against 64 bits.

Small whole numbers make every product and sum exact in fp32 (below 2^24), so that the result has to be the exact sum
rounded once, bit for bit.  With random numbers the sum of K products and the two terms behind it is off by at most
2 (K + 2) u of the sum of their magnitudes (u = 2^-24; 2 u a step for an accumulator that cuts off), then by eps / 2 of
the value for the last rounding."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(T, d, widths, dtype, whole, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if whole:
        rnd = lambda *s, std=1.0: torch.randint(-4, 5, s, generator=gen, device="cuda").to(TD[dtype])
    else:
        rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(TD[dtype])
    return {"H": [rnd(T, w) for w in widths], "W": [rnd(w, d, std=0.1) for w in widths], "b2": rnd(d), "R": rnd(T, d),
            "X": rnd(T, d)}


def exact(a, b2, R):
    K = sum(w.shape[0] for w in a["W"])
    y = R.double() + (a["b2"].double() if b2 else 0)
    size = R.double().abs() + (a["b2"].double().abs() if b2 else 0)
    for h, w in zip(a["H"], a["W"]):
        y = y + h.double() @ w.double()
        size = size + h.double().abs() @ w.double().abs()
    return y, 2 * (K + 2) * U * size


def check(Y, a, b2, R, whole):
    want, off = exact(a, b2, R)
    if whole:
        assert want.abs().max() < 2 ** 24
        assert torch.equal(Y, want.to(Y.dtype))
    else:
        assert ((Y.double() - want).abs() <= off + torch.finfo(Y.dtype).eps / 2 * (want.abs() + off)).all()


# tokens below, at and past a warp's 32 rows, a CTA's 128 and a pair's 256; widths below, at and past a tile
CASES = [(1, 8, [8]), (31, 72, [40, 136]), (128, 256, [64]), (257, 264, [8, 96, 264]), (300, 520, [128, 72]),
         (513, 1032, [256] * 4), (700, 40, [16] * 16)]


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d,widths", CASES)
def test_products(gpu_lib, T, d, widths, dtype, whole):
    a = make(T, d, widths, dtype, whole, seed=T)
    mlp = gpu_lib.ShardedMLP(T, d, widths, "gelu", dtype)
    for b2 in (True, False):
        Y = mlp.row_forward(a["H"], a["W"], b2=a["b2"] if b2 else None, residual=a["R"])
        check(Y, a, b2, a["R"], whole)
    plain = mlp.row_forward(a["H"], a["W"], b2=a["b2"])
    zero = mlp.row_forward(a["H"], a["W"], b2=a["b2"], residual=torch.zeros_like(a["R"]))
    assert torch.equal(plain, zero)
    mlp.check()
    proj = gpu_lib.ShardedAttentionProj(T, d, widths, widths, dtype)
    Z = proj.out_forward(a["W"], a["H"], residual=a["R"])
    check(Z, a, False, a["R"], whole)
    assert torch.equal(Z, mlp.row_forward(a["H"], a["W"], residual=a["R"]))
    proj.check()


@pytest.mark.parametrize("mode", ["ALWAYS", "BALANCE", "OFF"])
def test_schedules(gpu_lib, mode):
    """Tiles split along K: the residual is added once, by the part that finishes the tile."""
    T, d, widths = 700, 1160, [1024, 520, 512]
    a = make(T, d, widths, "bf16", True)
    mlp = gpu_lib.ShardedMLP(T, d, widths, "gelu", "bf16")
    proj = gpu_lib.ShardedAttentionProj(T, d, widths, widths, "bf16")
    for p in (mlp.plan, proj.plan):
        gpu_lib.tpmlp_plan_set_stream_k(p, getattr(gpu_lib, "STREAM_K_" + mode))
    check(mlp.row_forward(a["H"], a["W"], b2=a["b2"], residual=a["R"]), a, True, a["R"], True)
    assert bool(gpu_lib.tpmlp_last_split_tiles(gpu_lib.LAUNCH_FWD_ROW)) == (mode != "OFF")
    check(proj.out_forward(a["W"], a["H"], residual=a["R"]), a, False, a["R"], True)
    R = a["R"].clone()
    check(proj.out_forward(a["W"], a["H"], residual=R, out=R), a, False, a["R"], True)
    mlp.check()
    proj.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_place(gpu_lib, dtype):
    T, d, widths = 333, 328, [200, 72]
    a = make(T, d, widths, dtype, False)
    mlp = gpu_lib.ShardedMLP(T, d, widths, "gelu", dtype)
    want = mlp.row_forward(a["H"], a["W"], b2=a["b2"], residual=a["R"])
    R = a["R"].clone()
    assert mlp.row_forward(a["H"], a["W"], b2=a["b2"], residual=R, out=R) is R
    assert torch.equal(R, want)
    proj = gpu_lib.ShardedAttentionProj(T, d, widths, widths, dtype)
    R = a["R"].clone()
    assert torch.equal(proj.out_forward(a["W"], a["H"], residual=R, out=R),
                       proj.out_forward(a["W"], a["H"], residual=a["R"]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_whole_block(gpu_lib, act, dtype):
    """forward and forward_ckpt8 with a residual: what they keep is that of the calls without, Y the row product's."""
    T, d, widths = 203, 264, [72, 200, 136]
    a = make(T, d, widths, dtype, False)
    gen = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: (0.1 * torch.randn(*s, generator=gen, device="cuda")).to(TD[dtype])
    W1, b1 = [rnd(d, w) for w in widths], [rnd(w) for w in widths]
    W3, b3 = ([rnd(d, w) for w in widths], [rnd(w) for w in widths]) if act == "swiglu" else (None, None)
    mlp = gpu_lib.ShardedMLP(T, d, widths, act, dtype)
    kw = dict(b1_i=b1, b3_i=b3, b2=a["b2"])
    _, saved, H = mlp.forward(a["X"], W1, a["W"], W3, **kw)
    want = mlp.row_forward(H, a["W"], b2=a["b2"], residual=a["R"])
    Y, saved2, H2 = mlp.forward(a["X"], W1, a["W"], W3, residual=a["R"], **kw)
    assert torch.equal(Y, want)
    assert all(torch.equal(u, v) for u, v in zip(saved + H, saved2 + H2))
    _, ckpt = mlp.forward_ckpt8(a["X"], W1, a["W"], W3, **kw)
    R = a["R"].clone()
    buf = [torch.empty_like(c) for c in ckpt]
    Y, ckpt2 = mlp.forward_ckpt8(a["X"], W1, a["W"], W3, residual=R, out=(R, buf), **kw)
    assert torch.equal(Y, want) and Y is R
    unpack = lambda c, w: gpu_lib.ckpt8_unpack(c, T, w, dtype)
    n = 2 if act == "swiglu" else 1
    assert all(torch.equal(unpack(u, w), unpack(v, w)) for u, v, w in zip(ckpt, ckpt2, widths * n))
    mlp.check()


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_autograd(gpu_lib, act):
    """The gradients are those of the function without a residual, the residual's is dY; the same tensor as X and
    residual gets their sum."""
    T, d, widths = 96, 136, [72, 200]
    a = make(T, d, widths, "bf16", False)
    gen = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: (0.1 * torch.randn(*s, generator=gen, device="cuda")).bfloat16().requires_grad_()
    W = [rnd(d, w) for w in widths] + [rnd(w, d) for w in widths] + ([rnd(d, w) for w in widths] if act == "swiglu" else [])
    X, R = a["X"].requires_grad_(), a["R"].requires_grad_()
    dY = a["b2"].expand(T, d) + a["R"].detach()
    mlp = gpu_lib.ShardedMLP(T, d, widths, act, "bf16")
    want = torch.autograd.grad(gpu_lib.TPMLPCheckpointFunction.apply(mlp, X, *W), [X, *W], dY)
    got = torch.autograd.grad(gpu_lib.TPMLPResidualFunction.apply(mlp, X, R, *W), [X, *W, R], dY)
    assert all(torch.equal(u, v) for u, v in zip(want + (dY,), got))
    both = torch.autograd.grad(gpu_lib.TPMLPResidualFunction.apply(mlp, X, X, *W), X, dY)[0]
    assert torch.equal(both, want[0] + dY)
    with pytest.raises(ValueError, match="weights"):
        gpu_lib.TPMLPResidualFunction.apply(mlp, X, R, *W, W[0])


def test_bad_elements_of_the_residual_stay_where_they_are(gpu_lib):
    T, d, widths = 70, 72, [40]
    a = make(T, d, widths, "bf16", False)
    mlp = gpu_lib.ShardedMLP(T, d, widths, "gelu", "bf16")
    want = mlp.row_forward(a["H"], a["W"], residual=a["R"])
    R = a["R"].clone()
    R[3, 5], R[69, 71] = float("nan"), float("inf")
    got = mlp.row_forward(a["H"], a["W"], residual=R)
    assert torch.isnan(got[3, 5]) and got[69, 71] == float("inf")
    got[3, 5], got[69, 71] = want[3, 5], want[69, 71]
    assert torch.equal(got, want)


def test_past_32_bit_offsets(gpu_lib):
    """2.3e9 elements of residual and output; the last rows compared."""
    T, d = 140_000, 16384
    a = make(T, 8, [8], "bf16", True)
    W = torch.randint(-4, 5, (8, d), device="cuda").bfloat16()
    R = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    R[-300:] = torch.randint(-4, 5, (300, d), device="cuda").bfloat16()
    mlp = gpu_lib.ShardedMLP(T, d, [8], "gelu", "bf16")
    Y = mlp.row_forward(a["H"], [W], residual=R)
    for rows in (slice(0, 300), slice(131_000, 131_300), slice(T - 300, T)):
        want = a["H"][0][rows].double() @ W.double() + R[rows].double()
        assert torch.equal(Y[rows].double(), want.bfloat16().double())
    mlp.check()


def test_on_another_stream_and_in_a_graph(gpu_lib):
    T, d, widths = 300, 520, [128, 72]
    a = make(T, d, widths, "bf16", False)
    mlp = gpu_lib.ShardedMLP(T, d, widths, "gelu", "bf16")
    call = lambda **kw: mlp.row_forward(a["H"], a["W"], b2=a["b2"], residual=a["R"], **kw)
    want = call()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = call(stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    mlp.check()


def test_no_tokens(gpu_lib):
    mlp = gpu_lib.ShardedMLP(0, 64, [64], "gelu", "bf16")
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    assert mlp.row_forward([e(0, 64)], [e(64, 64)], residual=e(0, 64)).shape == (0, 64)
