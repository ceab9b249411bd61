"""8-bit checkpoints: pack and unpack byte for byte against the format's definition, and the MLP block's passes that
write and read them.

Exactness: packing rounds once, from values the reference has exactly, so every byte is compared for equality.  The
block's forward pass differs from tpmlp_forward only in what it keeps, its backward pass from
tpmlp_backward_recompute on the unpacked checkpoints only in where it reads them: both are compared bit for bit."""
import numpy as np
import pytest
import torch

import operators_reference as ref
import synthetic_inputs as si
from gpu_helpers import cat_cols, cat_rows, rel_err, to_np, tol_for

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


def values_of(buf, rows, cols):
    return ref.values(*ref.split(buf.cpu().numpy(), rows, cols), cols)


def check_pack(tp, x, x_in=None):
    """Pack x (numpy gives the same numbers), compare the bytes; unpack, compare the values.  Returns the buffer."""
    x_in = x if x_in is None else x_in
    rows, cols = x.shape
    buf = torch.full((tp.tpmlp_ckpt8_size(rows, cols),), 0xA5, dtype=torch.uint8, device="cuda")
    assert buf.numel() == ref.nbytes(rows, cols)
    tp.ckpt8_pack(x_in, out=buf)
    codes, scale = ref.split(buf.cpu().numpy(), rows, cols)
    want_codes, want_scale = ref.pack(x.double().cpu().numpy())
    assert np.array_equal(scale, want_scale)
    fine = scale != 255
    # a zero may carry either sign of the input; the sign bit is the input's
    assert np.array_equal(codes[fine], want_codes[fine])
    assert (ref.pad_bytes(buf.cpu().numpy(), rows, cols) == 0xA5).all()
    dtype = "bf16" if x.dtype == torch.bfloat16 else "fp32"
    out = tp.ckpt8_unpack(buf, rows, cols, dtype)
    want = ref.values(want_codes, want_scale, cols)
    assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)
    again = tp.ckpt8_unpack(tp.ckpt8_pack(out), rows, cols, dtype)
    assert np.array_equal(again.double().cpu().numpy(), want, equal_nan=True)
    return buf


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 16), (3, 24), (32, 64), (33, 72), (31, 128), (100, 136), (257, 1000),
                                       (2048, 512)])
def test_pack_unpack(gpu_lib, rows, cols, dtype):
    gen = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=gen) * torch.exp(3 * torch.randn(cols, generator=gen))
    check_pack(gpu_lib, x.to(TD[dtype]).cuda())


def test_pack_fp32_odd_width(gpu_lib):
    """fp32 widths are multiples of 4: groups that end after 4 or 12 columns."""
    for cols in (4, 12, 20, 44):
        check_pack(gpu_lib, torch.randn(50, cols).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pack_special_values(gpu_lib, dtype):
    big = torch.finfo(TD[dtype]).max
    tiny = torch.finfo(TD[dtype]).tiny
    x = torch.zeros(64, 64, dtype=torch.float64)
    x[1] = 1.0
    x[2, 5], x[3, 5], x[4, 17] = float("nan"), float("inf"), float("-inf")
    x[5], x[6, 3], x[7] = big, -big, tiny
    x[8, 0], x[8, 1:] = big, 1.0
    x[9] = torch.linspace(0.9, 1.0, 64, dtype=torch.float64) * big
    for i in range(8):  # the largest magnitude at, just below and just above 448 * 2^e
        m = 448.0 * 2.0 ** (20 * i - 70)
        step = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -22
        x[10 + i, :16] = m * torch.linspace(-1, 1, 16, dtype=torch.float64)
        x[10 + i, 16:32] = x[10 + i, :16] / (1 + step)
        x[10 + i, 32:48] = x[10 + i, :16] * (1 + step)
    x[20, :16] = torch.arange(16) * 0.0625 + 16  # ties between codes: 3 bits behind the leading one
    x[21, :16] = (torch.arange(16) + 0.5) * 2.0 ** -9
    x[21, 15] = 1.0
    x[22, :16] = (torch.arange(16) + 0.5) * 2.0 ** -9 / 448
    x[22, 15] = 1.0
    x[23, :16] = -x[20, :16]
    x[24, :16] = tiny * torch.arange(16) / 4  # below the smallest scale's numbers
    x[25, :16] = 2.0 ** -118 * torch.arange(16)
    x[26, :16] = -0.0
    check_pack(gpu_lib, x.to(TD[dtype]).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pack_strided(gpu_lib, dtype):
    """A column slice of a wider tensor in, and out again into another: the neighbours stay as they are."""
    wide = torch.randn(45, 96).to(TD[dtype]).cuda()
    part = wide[:, 16:64]
    buf = check_pack(gpu_lib, part.contiguous(), part)
    out = torch.full((45, 80), 7.0, dtype=TD[dtype], device="cuda")
    gpu_lib.ckpt8_unpack(buf, 45, 48, dtype, out=out[:, 8:56])
    assert np.array_equal(out[:, 8:56].double().cpu().numpy(), values_of(buf, 45, 48))
    assert (out[:, :8] == 7).all() and (out[:, 56:] == 7).all()


def test_pack_past_32_bits(gpu_lib):
    """A tensor of more than 2^32 bytes: its last rows, against the same rows packed alone."""
    rows, cols = 65600, 32768
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    buf = gpu_lib.ckpt8_pack(x)
    last = 64 + 32
    n = -(-rows // 32) * 2048
    tail = gpu_lib.ckpt8_pack(x[-last:].contiguous())
    B = last // 32
    assert torch.equal(buf[: n * 512][-B * 2048 * 512:], tail[: B * 2048 * 512])
    assert torch.equal(buf[n * 512:][-B * 2048 * 32:], tail[B * 2048 * 512:])
    out = gpu_lib.ckpt8_unpack(buf, rows, cols)
    assert torch.equal(out[-last:], gpu_lib.ckpt8_unpack(tail, last, cols))


# ---------------------------------------------------------------- the block's passes

def setup(tp, T, d, d_i, act, dtype, seed=5, bias=True, stream_k=None):
    inp = si.make_inputs(T, d, d_i, act, dtype, seed=seed)
    mlp = tp.ShardedMLP(T, d, d_i, act, dtype)
    if stream_k is not None:
        tp.tpmlp_plan_set_stream_k(mlp.plan, stream_k)
    cu = lambda xs: [x.cuda() for x in xs] if xs is not None else None
    s = {"X": inp.X.cuda(), "dY": inp.dY.cuda(), "W1": cu(inp.W1_i), "W2": cu(inp.W2_i), "W3": cu(inp.W3_i), "b": {}}
    if bias:
        b = si.make_biases(d, d_i, act, dtype, seed=seed)
        s["b"] = dict(b1_i=cu(b["b1_i"]), b3_i=cu(b["b3_i"]) if act == "swiglu" else None, b2=b["b2"].cuda())
    return mlp, s


CASES = [  # T, d, d_i
    (333, 200, (8, 96, 264, 152)),  # widths that end inside a group, a block and a tile
    (1, 64, (16,)), (32, 64, (128, 128)), (300, 1104, (264, 40)),
    (700, 2048, (512, 24)),  # K of more than 1024: the 8-warp epilogues
]


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("stream_k", [None, 2])
@pytest.mark.parametrize("T,d,d_i", CASES)
def test_forward_and_backward_bits(gpu_lib, T, d, d_i, act, dtype, stream_k):
    """Y as tpmlp_forward gives it; the checkpoints those of the pre-activations; every gradient as
    tpmlp_backward_recompute gives it for the kept values."""
    tp = gpu_lib
    mlp, s = setup(tp, T, d, d_i, act, dtype, stream_k=stream_k)
    Y, saved, H = mlp.forward(s["X"], s["W1"], s["W2"], s["W3"], **s["b"])
    bufs = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in mlp.ckpt8_sizes()]
    Y8, ckpt = mlp.forward_ckpt8(s["X"], s["W1"], s["W2"], s["W3"], out=(torch.empty_like(Y), bufs), **s["b"])
    torch.cuda.synchronize()
    mlp.check()
    assert torch.equal(Y, Y8)
    n = len(d_i)
    kept = []
    for i, (c, a) in enumerate(zip(ckpt, saved)):
        w = d_i[i % n]
        if dtype == "fp32":  # saved is the accumulator itself
            codes, scale = ref.split(c.cpu().numpy(), T, w)
            want = ref.pack(to_np(a))
            assert np.array_equal(codes, want[0]) and np.array_equal(scale, want[1])
        else:  # saved is the accumulator rounded to bf16, off by 2^-8 of it
            v, a64 = values_of(c, T, w), to_np(a)
            g = np.zeros((T, -(-w // 16) * 16))
            g[:, :w] = np.abs(a64)
            m = np.repeat(g.reshape(T, -1, 16).max(-1), 16, 1)[:, :w] * (1 + 2.0 ** -7)
            # a code is off by 2^-4 of its value, or half of 2^-9 2^e with 2^e <= m / 224
            assert (np.abs(v - a64) <= np.abs(a64) * (1 + 2.0 ** -7) * (2.0 ** -4 + 2.0 ** -8) + 2.0 ** -10 * m / 224).all()
        assert (ref.pad_bytes(c.cpu().numpy(), T, w) == 0xA5).all()
        kept.append(tp.ckpt8_unpack(c, T, w, dtype))
        assert np.array_equal(to_np(kept[-1]), values_of(c, T, w))
    want = mlp.backward(s["X"], s["W1"], s["W2"], kept, [torch.empty_like(h) for h in H], s["dY"], s["W3"],
                        bias_grads=True, recompute=True)
    got = mlp.backward_ckpt8(s["X"], s["W1"], s["W2"], ckpt, s["dY"], s["W3"], bias_grads=True)
    torch.cuda.synchronize()
    mlp.check()
    for k in ("dX", "dW1", "dW2", "db1", "db2") + (("dW3", "db3") if act == "swiglu" else ()):
        a, b = (x if isinstance(x, list) else [x] for x in (want[k], got[k]))
        for i, (x, y) in enumerate(zip(a, b)):
            assert torch.equal(x, y), (k, i)


def test_checkpoints_of_exact_sums(gpu_lib):
    """Small integers: the accumulators are bf16 numbers, so the bf16 path's checkpoints can be compared byte for
    byte.  |A| <= 64 * 2 * 2 = 256 and whole."""
    tp = gpu_lib
    T, d, d_i = 290, 64, (72, 256, 24)
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randint(-2, 3, s, generator=gen).to(torch.bfloat16).cuda()
    for act in ("gelu", "swiglu"):
        mlp = tp.ShardedMLP(T, d, d_i, act, "bf16")
        X, W1, W3 = rnd(T, d), [rnd(d, w) for w in d_i], [rnd(d, w) for w in d_i]
        W2 = [rnd(w, d) for w in d_i]
        _, ckpt = mlp.forward_ckpt8(X, W1, W2, W3 if act == "swiglu" else None)
        for W, cs in ((W1, ckpt[:3]), (W3, ckpt[3:])):
            for w, c in zip(W, cs):
                codes, scale = ref.split(c.cpu().numpy(), T, w.shape[1])
                want = ref.pack((X.double() @ w.double()).cpu().numpy())
                assert np.array_equal(codes, want[0]) and np.array_equal(scale, want[1])


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_against_the_formula(gpu_lib, act, dtype):
    """The gradients of the kept values, in 64 bits; the framework's tolerances."""
    tp = gpu_lib
    T, d, d_i = (260, 136, (40, 264)) if dtype == "bf16" else (45, 36, (20, 44))
    mlp, s = setup(tp, T, d, d_i, act, dtype)
    _, ckpt = mlp.forward_ckpt8(s["X"], s["W1"], s["W2"], s["W3"], **s["b"])
    g = mlp.backward_ckpt8(s["X"], s["W1"], s["W2"], ckpt, s["dY"], s["W3"], bias_grads=True)
    n = len(d_i)
    kept = [torch.from_numpy(values_of(c, T, d_i[i % n])) for i, c in enumerate(ckpt)]
    A, Uk = torch.cat(kept[:n], 1), torch.cat(kept[n:], 1) if act == "swiglu" else None
    X, dY = s["X"].double().cpu(), s["dY"].double().cpu()
    W1, W2 = (torch.cat([w.double().cpu() for w in s[k]], dim) for k, dim in (("W1", 1), ("W2", 0)))
    dH = dY @ W2.T
    if act == "swiglu":
        W3 = torch.cat([w.double().cpu() for w in s["W3"]], 1)
        sg = torch.sigmoid(A)
        H, dU, dA = Uk * A * sg, dH * A * sg, dH * Uk * sg * (1 + A * (1 - sg))
        dX = dA @ W1.T + dU @ W3.T
    else:
        cdf = 0.5 * torch.erfc(-A / 2 ** 0.5)
        H, dA = A * cdf, dH * (cdf + A * torch.exp(-A * A / 2) / (2 * np.pi) ** 0.5)
        dX = dA @ W1.T
    errs = {"dX": rel_err(to_np(g["dX"]), dX.numpy()), "dW1": rel_err(cat_cols(g["dW1"]), (X.T @ dA).numpy()),
            "dW2": rel_err(cat_rows(g["dW2"]), (H.T @ dY).numpy()), "db2": rel_err(to_np(g["db2"]), dY.sum(0).numpy()),
            "db1": rel_err(np.concatenate([to_np(x) for x in g["db1"]]), dA.sum(0).numpy())}
    if act == "swiglu":
        errs["dW3"] = rel_err(cat_cols(g["dW3"]), (X.T @ dU).numpy())
        errs["db3"] = rel_err(np.concatenate([to_np(x) for x in g["db3"]]), dU.sum(0).numpy())
    bad = {k: v for k, v in errs.items() if not v <= tol_for(dtype)}
    assert not bad, f"{bad} of {errs}"


def test_sixteen_shards(gpu_lib):
    """The largest tables (SwiGLU, t = 16): dW2 gets a launch of its own."""
    tp = gpu_lib
    mlp, s = setup(tp, 150, 48, (8, 16, 8, 24, 8, 8, 16, 8, 8, 8, 32, 8, 8, 16, 8, 8), "swiglu", "bf16")
    Y, saved, H = mlp.forward(s["X"], s["W1"], s["W2"], s["W3"], **s["b"])
    Y8, ckpt = mlp.forward_ckpt8(s["X"], s["W1"], s["W2"], s["W3"], **s["b"])
    assert torch.equal(Y, Y8)
    kept = [tp.ckpt8_unpack(c, 150, w) for c, w in zip(ckpt, mlp.plan.d_i * 2)]
    want = mlp.backward(s["X"], s["W1"], s["W2"], kept, H, s["dY"], s["W3"], recompute=True)
    got = mlp.backward_ckpt8(s["X"], s["W1"], s["W2"], ckpt, s["dY"], s["W3"])
    for k in ("dW1", "dW2", "dW3"):
        assert all(torch.equal(x, y) for x, y in zip(want[k], got[k])), k
    assert torch.equal(want["dX"], got["dX"])


def test_infinite_and_nan_inputs(gpu_lib):
    """A token with an infinity spoils its own row of the checkpoint, in every group, and no other."""
    tp = gpu_lib
    mlp, s = setup(tp, 70, 64, (48,), "gelu", "bf16", bias=False)
    clean = mlp.forward_ckpt8(s["X"], s["W1"], s["W2"])[1][0]
    s["X"][11, 3] = float("inf")
    s["X"][40, 9] = float("nan")
    got = mlp.forward_ckpt8(s["X"], s["W1"], s["W2"])[1][0]
    a, b = values_of(clean, 70, 48), values_of(got, 70, 48)
    rows = np.ones(70, bool)
    rows[[11, 40]] = False
    assert np.array_equal(a[rows], b[rows])
    assert np.isnan(b[[11, 40]]).all()


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_autograd_function(gpu_lib, act):
    tp = gpu_lib
    mlp, s = setup(tp, 130, 64, (40, 64), act, "bf16", bias=False)
    ws = s["W1"] + s["W2"] + (s["W3"] if act == "swiglu" else [])
    leaves = [x.clone().requires_grad_() for x in [s["X"]] + ws]
    Y = tp.TPMLPCheckpointFunction.apply(mlp, *leaves)
    Y.backward(s["dY"])
    Y8, ckpt = mlp.forward_ckpt8(s["X"], s["W1"], s["W2"], s["W3"])
    g = mlp.backward_ckpt8(s["X"], s["W1"], s["W2"], ckpt, s["dY"], s["W3"])
    want = [g["dX"]] + g["dW1"] + g["dW2"] + (g["dW3"] if act == "swiglu" else [])
    assert torch.equal(Y, Y8)
    for x, w in zip(leaves, want):
        assert torch.equal(x.grad, w)


def test_other_stream_and_capture(gpu_lib):
    tp = gpu_lib
    mlp, s = setup(tp, 200, 128, (96, 64), "swiglu", "bf16", bias=False)
    step = lambda **kw: (lambda Yc: (Yc, mlp.backward_ckpt8(s["X"], s["W1"], s["W2"], Yc[1], s["dY"], s["W3"], **kw)))(
        mlp.forward_ckpt8(s["X"], s["W1"], s["W2"], s["W3"], **kw))
    (Y, ckpt), g = step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    (Y2, _), g2 = step(stream=st)
    st.synchronize()
    assert torch.equal(Y, Y2) and torch.equal(g["dX"], g2["dX"]) and torch.equal(g["dW2"][1], g2["dW2"][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (Y3, _), g3 = step()
        kept = tp.ckpt8_unpack(tp.ckpt8_pack(s["X"]), 200, 128)
    s["X"].copy_(s["X"].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    (Y, _), g = step()
    assert torch.equal(Y, Y3) and torch.equal(g["dX"], g3["dX"]) and torch.equal(g["dW1"][0], g3["dW1"][0])
    assert np.array_equal(to_np(kept), ref.values(*ref.pack(to_np(s["X"])), 128))
    mlp.check()


def test_empty(gpu_lib):
    tp = gpu_lib
    mlp, s = setup(tp, 0, 64, (32, 16), "gelu", "bf16", bias=False)
    Y, ckpt = mlp.forward_ckpt8(s["X"], s["W1"], s["W2"])
    g = mlp.backward_ckpt8(s["X"], s["W1"], s["W2"], ckpt, s["dY"], bias_grads=True)
    assert Y.shape == (0, 64) and all(not x.any() for x in g["dW1"] + g["dW2"] + g["db1"] + [g["db2"]])
    x = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    assert tp.ckpt8_unpack(tp.ckpt8_pack(x), 0, 16).shape == (0, 16)


def test_python_refusals(gpu_lib):
    """Wrong shapes, types, strides and devices are refused before any launch."""
    tp = gpu_lib
    mlp, s = setup(tp, 40, 64, (32, 16), "swiglu", "bf16", bias=False)
    _, ckpt = mlp.forward_ckpt8(s["X"], s["W1"], s["W2"], s["W3"])
    ok = dict(X=s["X"], W1_i=s["W1"], W2_i=s["W2"], W3_i=s["W3"])
    for kw in (dict(X=s["X"][:39]), dict(X=s["X"].float()), dict(X=s["X"].cpu()), dict(W1_i=s["W1"][:1]),
               dict(W3_i=None), dict(W2_i=s["W1"]), dict(b1_i=[torch.zeros(32, device="cuda")] * 2),
               dict(W1_i=[w.t().contiguous().t() for w in s["W1"]])):
        with pytest.raises(ValueError):
            mlp.forward_ckpt8(**{**ok, **kw})
    for kw in (dict(ckpt=ckpt[:3]), dict(ckpt=[c[:-1] for c in ckpt]), dict(ckpt=[c.short() for c in ckpt]),
               dict(dY=s["dY"][:3])):
        with pytest.raises(ValueError):
            mlp.backward_ckpt8(**{**ok, **dict(ckpt=ckpt, dY=s["dY"]), **kw})
    x = torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda")
    for y in (x.t(), x.half(), x[0], x.expand(8, 32)[:, ::2]):
        with pytest.raises(ValueError):
            tp.ckpt8_pack(y)
    with pytest.raises(tp.TpmlpError):
        tp.ckpt8_pack(x[:1].expand(8, 32))  # rows on top of one another
    with pytest.raises(tp.TpmlpError):
        tp.ckpt8_pack(x[:, 1:17])  # not on a 16-byte boundary
    buf = tp.ckpt8_pack(x)
    # (9 rows have the same size as 8: nothing can tell those apart)
    for kw in (dict(rows=33), dict(cols=48), dict(out=x[:, :16]), dict(out=x.float())):
        with pytest.raises(ValueError):
            tp.ckpt8_unpack(**{**dict(ckpt=buf, rows=8, cols=32), **kw})


def test_block_past_32_bits(gpu_lib):
    """Checkpoints and activations of more than 2^32 bytes: the last tokens' Y, checkpoint and dX, against the same
    tokens alone (a row's sums do not depend on how many rows there are; K of 36 blocks, no stream-K)."""
    tp = gpu_lib
    free, _ = torch.cuda.mem_get_info()
    if free < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    T, d, w, last = 1 << 20, 64, 4608, 96
    gen = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).bfloat16()
    X, dY, W1, W2 = rnd(T, d), rnd(T, d), [rnd(d, w, std=0.1)], [rnd(w, d, std=0.02)]
    whole, part = tp.ShardedMLP(T, d, [w]), tp.ShardedMLP(last, d, [w])
    for m in (whole, part):
        tp.tpmlp_plan_set_stream_k(m.plan, tp.STREAM_K_OFF)
    Y, ckpt = whole.forward_ckpt8(X, W1, W2)
    Yp, cp = part.forward_ckpt8(X[-last:].contiguous(), W1, W2)
    assert ckpt[0].numel() > 1 << 32
    assert torch.equal(Y[-last:], Yp)
    codes, tail = T * w, last * w  # whole blocks of rows and columns
    assert torch.equal(ckpt[0][:codes][-tail:], cp[0][:tail])
    assert torch.equal(ckpt[0][codes:][-tail // 16:], cp[0][tail:])
    dX = whole.backward_ckpt8(X, W1, W2, ckpt, dY)["dX"]
    assert torch.equal(dX[-last:], part.backward_ckpt8(X[-last:].contiguous(), W1, W2, cp, dY[-last:].contiguous())["dX"])
    whole.check()
