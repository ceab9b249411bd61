"""Cases for measuring the operators that stand next to the library's GEMM launches in a training step.

qk_fwd, qk_bwd  norm of each query and key head and position rotation in one pass over the shards' fused QKV
                buffers, and its backward pass (tpmlp_attn_qk_norm_rope_*)
keep            a tensor kept in 8 bits between two passes: packed, then unpacked (tpmlp_ckpt8_pack / _unpack)
mlp_step        forward and backward of the sharded MLP block with 8-bit activation checkpoints
                (tpmlp_forward_ckpt8, tpmlp_backward_ckpt8)
mlp_bwd         the backward pass alone, from a checkpoint written earlier

`own` chooses between the plain form (elementary torch operations in 32 bits) and the library's kernels.

8-bit checkpoint of a [rows x cols] tensor: groups of 16 columns of a row; m the largest magnitude of a group; its
scale is 2^e with the smallest e for which m <= 448 * 2^e, within [-117, 120]; an element is kept as the nearest
e4m3 number (ties to even) to x * 2^-e.  Storage: blocks of 32 rows x 16 columns, 512 bytes each, row-major, then the
scale bytes e + 127, 32 per block in the blocks' order.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _w(text):
    return [int(v) for v in text.split(",")]


def listed():
    heads8 = ",".join(["2048"] * 8)
    kv8 = ",".join(["128"] * 8)
    w96 = ",".join(["384"] * 8)
    return [
        # one new token: 16 query heads and one key head of 128 on each of 8 shards; latency counts
        {"name": "qk_fwd token", "op": "qk_fwd", "T": 1, "dq": heads8, "dkv": kv8, "D": 128, "R": 128,
         "layout": "halves", "dtype": "bf16"},
        # the GPT-2 8.3B attention shape: 8 shards of four heads of 96, a training batch of 8 x 2048 tokens
        {"name": "qk_fwd batch", "op": "qk_fwd", "T": 16384, "dq": w96, "dkv": w96, "D": 96, "R": 96,
         "layout": "halves", "dtype": "bf16"},
        # unequal shards, part of each head rotated, neighbouring pairs, an odd number of tokens, fp32
        {"name": "qk_fwd ragged", "op": "qk_fwd", "T": 1533, "dq": "640,384", "dkv": "128,64", "D": 64, "R": 32,
         "layout": "pairs", "dtype": "fp32"},
        # backward of the training batch
        {"name": "qk_bwd batch", "op": "qk_bwd", "T": 16384, "dq": w96, "dkv": w96, "D": 96, "R": 96,
         "layout": "halves", "dtype": "bf16"},
        # backward of an odd batch with grouped key heads, fp32
        {"name": "qk_bwd ragged", "op": "qk_bwd", "T": 777, "dq": "1024,512", "dkv": "128,128", "D": 128, "R": 64,
         "layout": "halves", "dtype": "fp32"},
        # a layer's input of 8192 tokens kept between the passes
        {"name": "keep batch", "op": "keep", "T": 8192, "w": 4096, "dtype": "bf16"},
        # odd sizes: a last block of rows and a last group of columns that are not full
        {"name": "keep ragged", "op": "keep", "T": 1531, "w": 1364, "dtype": "fp32"},
        # the Llama-style SwiGLU block, 8 shards
        {"name": "mlp_step swiglu", "op": "mlp_step", "T": 8192, "d": 4096, "widths": ",".join(["1376"] * 8),
         "act": "swiglu", "bias": False, "dtype": "bf16"},
        # the GPT-2-small block with its biases, 4 shards
        {"name": "mlp_step gelu", "op": "mlp_step", "T": 8192, "d": 768, "widths": "768,768,768,768",
         "act": "gelu", "bias": True, "dtype": "bf16"},
        # a short batch, unequal shards whose widths end inside a group
        {"name": "mlp_step ragged", "op": "mlp_step", "T": 203, "d": 264, "widths": "72,200,136", "act": "swiglu",
         "bias": True, "dtype": "bf16"},
        # backward alone, unequal shards
        {"name": "mlp_bwd gelu", "op": "mlp_bwd", "T": 8192, "d": 2048, "widths": "1536,2560,2048,2048",
         "act": "gelu", "bias": False, "dtype": "bf16"},
        # the smallest block, fp32 storage
        {"name": "mlp_bwd fp32", "op": "mlp_bwd", "T": 32, "d": 64, "widths": "128,128", "act": "gelu",
         "bias": True, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "keep", "mlp_step", "mlp_bwd"])
    if op in ("qk_fwd", "qk_bwd"):
        D = rng.choice([32, 64, 80, 96, 128, 160, 192, 256])
        t = rng.randint(1, 8)
        heads = [rng.randint(1, 16) for _ in range(t)]
        kv = [max(1, h // rng.choice([1, 2, 4, 8])) for h in heads]
        most = 16384 * 8 * 768 // (D * (sum(heads) + sum(kv)))
        return {"op": op, "T": _log(rng, 1, min(16384, most)), "dq": ",".join(str(D * h) for h in heads),
                "dkv": ",".join(str(D * h) for h in kv), "D": D, "R": rng.choice([D, D, D // 2, D // 4 // 2 * 2]),
                "layout": rng.choice(["halves", "pairs"]), "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "keep":
        return {"op": op, "T": _log(rng, 1, 8192), "w": 8 * _log(rng, 1, 512), "dtype": rng.choice(["bf16", "fp32"])}
    if op == "mlp_bwd" and rng.random() < 0.5:  # fp32 storage: small blocks
        return {"op": op, "T": _log(rng, 16, 256), "d": 4 * rng.randint(8, 64),
                "widths": ",".join(str(4 * rng.randint(4, 64)) for _ in range(rng.randint(1, 4))),
                "act": rng.choice(["gelu", "swiglu"]), "bias": rng.random() < 0.5, "dtype": "fp32"}
    return {"op": op, "T": _log(rng, 16, 8192), "d": 8 * _log(rng, 16, 512),
            "widths": ",".join(str(8 * _log(rng, 8, 172)) for _ in range(rng.randint(1, 8))),
            "act": rng.choice(["gelu", "swiglu"]), "bias": rng.random() < 0.5, "dtype": "bf16"}


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    T = case["T"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)

    if case["op"] in ("qk_fwd", "qk_bwd"):
        dq, dkv, D = _w(case["dq"]), _w(case["dkv"]), case["D"]
        s = {"QKV": [normal(T, q + 2 * k) for q, k in zip(dq, dkv)],
             "gq": (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt),
             "gk": (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)}
        # sequences of up to 2048 tokens behind one another, the last ones far into a long context
        first = torch.randint(0, 1 << 17, (1,), generator=gen, device="cuda")
        s["pos"] = torch.arange(T, device="cuda") % 2048 + first
        if case["op"] == "qk_bwd":
            s["dQK"] = [normal(T, q + k) for q, k in zip(dq, dkv)]
            s["dV"] = [normal(T, k) for k in dkv]
        return s
    if case["op"] == "keep":  # activations: columns of different sizes, some of them large
        col = torch.exp(torch.randn(case["w"], generator=gen, device="cuda"))
        return {"x": (torch.randn(T, case["w"], generator=gen, device="cuda") * col).to(dt)}
    widths, d = _w(case["widths"]), case["d"]
    s = {"X": normal(T, d), "dY": normal(T, d), "W1": [normal(d, w, std=0.02) for w in widths],
         "W2": [normal(w, d, std=0.02) for w in widths],
         "W3": [normal(d, w, std=0.02) for w in widths] if case["act"] == "swiglu" else None,
         "b1": [normal(w, std=0.1) for w in widths] if case["bias"] else None,
         "b3": [normal(w, std=0.1) for w in widths] if case["bias"] and case["act"] == "swiglu" else None,
         "b2": normal(d, std=0.1) if case["bias"] else None}
    if case["op"] == "mlp_bwd":  # pre-activations of the size that W1 gives them, kept by an earlier forward pass
        std = max(0.05, 0.02 * math.sqrt(d))
        n = 2 if case["act"] == "swiglu" else 1
        s["ckpt"] = [_store(torch.randn(T, w, generator=gen, device="cuda") * std) for w in widths * n]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:  # the plan and its workspace, which a program keeps
        import megatron_tensor_transformer_column_gb300 as tp

        s["tp"] = tp
        if case["op"] in ("qk_fwd", "qk_bwd"):
            dq, dkv = _w(case["dq"]), _w(case["dkv"])
            s["proj"] = tp.ShardedAttentionProj(case["T"], 1024, dq, dkv, case["dtype"])
            s["proj"].set_qk_norm_rope(case["D"], case["R"], layout=case["layout"], eps=1e-6, base=10000.0)
        elif case["op"] != "keep":
            s["mlp"] = tp.ShardedMLP(case["T"], case["d"], _w(case["widths"]), case["act"], case["dtype"])
    return s


# ------------------------------------------------------------------ 8-bit numbers, plain form

def _quantise(x):
    """[rows x cols] fp32 -> (codes as e4m3 [rows x G x 16], exponents [rows x G])."""
    rows, cols = x.shape
    g = torch.nn.functional.pad(x, (0, -cols % 16)).view(rows, -1, 16)
    m = g.abs().amax(-1)
    man, ex = torch.frexp(m)  # m = man * 2^ex, man in [0.5, 1)
    e = torch.where(m > 0, ex - 9 + (man > 0.875).int(), torch.full_like(ex, -117)).clamp(-117, 120)
    return torch.ldexp(g, -e[..., None]).to(torch.float8_e4m3fn), e


def _values(codes, e, cols):
    return torch.ldexp(codes.float(), e[..., None]).flatten(1)[:, :cols]


def _store(x):
    """A checkpoint as it lies in memory: blocks of 32 x 16 codes, then the scale bytes."""
    codes, e = _quantise(x)
    rows, G = e.shape
    pad = -rows % 32
    c = torch.nn.functional.pad(codes.view(torch.uint8), (0, 0, 0, 0, 0, pad)).view(-1, 32, G, 16).transpose(1, 2)
    b = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, 0, 0, pad)).view(-1, 32, G).transpose(1, 2)
    return torch.cat([c.reshape(-1), b.reshape(-1)])


def _load(buf, rows, cols):
    G, B = -(-cols // 16), -(-rows // 32)
    n = B * G * 512
    c = buf[:n].view(torch.float8_e4m3fn).view(B, G, 32, 16).transpose(1, 2).reshape(B * 32, G, 16)
    e = buf[n:].view(B, G, 32).transpose(1, 2).reshape(B * 32, G).int() - 127
    return _values(c, e, cols)[:rows]


# ------------------------------------------------------------------ plain forms

def _angles(s, case):
    R = case["R"]
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    phi = s["pos"].double()[:, None] * f
    return phi.cos().float()[:, None], phi.sin().float()[:, None]  # [T x 1 x R/2]


def _rotate(x, cos, sin, R, layout):
    r, rest = x[..., :R], x[..., R:]
    if layout == "halves":
        a, b = r[..., : R // 2], r[..., R // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _heads(xs, widths, offsets, D):
    """The shards' columns [offset, offset + width) side by side, as [T x heads x D] in 32 bits."""
    return torch.cat([x[:, o:o + w] for x, w, o in zip(xs, widths, offsets)], 1).float().unflatten(1, (-1, D))


def _join(q, k, dq, dkv, more=None, dt=None):
    q, k = q.flatten(1).to(dt).split(dq, 1), k.flatten(1).to(dt).split(dkv, 1)
    return [torch.cat(c, 1) for c in (zip(q, k) if more is None else zip(q, k, more))]


def _plain_qk_fwd(s, case):
    dq, dkv, D = _w(case["dq"]), _w(case["dkv"]), case["D"]
    cos, sin = _angles(s, case)

    def side(x, g):
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        return _rotate(n * g.float(), cos, sin, case["R"], case["layout"])

    q = side(_heads(s["QKV"], dq, [0] * len(dq), D), s["gq"])
    k = side(_heads(s["QKV"], dkv, dq, D), s["gk"])
    return _join(q, k, dq, dkv, dt=DTYPES[case["dtype"]])


def _plain_qk_bwd(s, case):
    dq, dkv, D, dt = _w(case["dq"]), _w(case["dkv"]), case["D"], DTYPES[case["dtype"]]
    cos, sin = _angles(s, case)

    def side(x, dy, g):
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        n = x * r
        w = _rotate(dy, cos, -sin, case["R"], case["layout"])
        dg = (w * n).sum((0, 1))
        w = w * g.float()
        return r * (w - n * (w * n).mean(-1, keepdim=True)), dg.to(dt)

    q, dgq = side(_heads(s["QKV"], dq, [0] * len(dq), D), _heads(s["dQK"], dq, [0] * len(dq), D), s["gq"])
    k, dgk = side(_heads(s["QKV"], dkv, dq, D), _heads(s["dQK"], dkv, dq, D), s["gk"])
    return {"dQKV": _join(q, k, dq, dkv, s["dV"], dt), "dgq": dgq, "dgk": dgk}


def _phi(a):
    return 0.5 * (1 + torch.erf(a / math.sqrt(2)))


def _cat(xs, dim):
    return torch.cat(xs, dim).float()


def _plain_mlp(s, case):
    sw, dt, widths, T = case["act"] == "swiglu", DTYPES[case["dtype"]], _w(case["widths"]), case["T"]
    out = {}
    X, dY, W1, W2 = s["X"].float(), s["dY"].float(), _cat(s["W1"], 1), _cat(s["W2"], 0)
    W3 = _cat(s["W3"], 1) if sw else None
    if case["op"] == "mlp_step":
        A = X @ W1 if s["b1"] is None else X @ W1 + _cat(s["b1"], 0)
        if sw:
            U = X @ W3 if s["b3"] is None else X @ W3 + _cat(s["b3"], 0)
            H = U * A * torch.sigmoid(A)
        else:
            H = A * _phi(A)
        Y = H @ W2 if s["b2"] is None else H @ W2 + s["b2"].float()
        out["Y"] = Y.to(dt)

        def keep(x):  # each shard's tensor is kept by itself
            return torch.cat([_values(*_quantise(v), w) for v, w in zip(x.split(widths, 1), widths)], 1)

        A = keep(A)
        U = keep(U) if sw else None
    else:
        got = [_load(b, T, w) for b, w in zip(s["ckpt"], widths * (2 if sw else 1))]
        A = torch.cat(got[: len(widths)], 1)
        U = torch.cat(got[len(widths):], 1) if sw else None
    dH = dY @ W2.T
    if sw:
        sg = torch.sigmoid(A)
        H = U * A * sg
        dA, dU = dH * U * (sg + A * sg * (1 - sg)), dH * A * sg
    else:
        p = _phi(A)
        H = A * p
        dA = dH * (p + A * torch.exp(-0.5 * A * A) / math.sqrt(2 * math.pi))
    out["dW2"] = list((H.T @ dY).to(dt).split(widths, 0))
    out["dW1"] = list((X.T @ dA).to(dt).split(widths, 1))
    dX = dA @ W1.T
    if sw:
        out["dW3"] = list((X.T @ dU).to(dt).split(widths, 1))
        dX = dX + dU @ W3.T
    out["dX"] = dX.to(dt)
    if case["bias"]:
        out["db2"] = dY.sum(0).to(dt)
        out["db1"] = list(dA.sum(0).to(dt).split(widths))
        if sw:
            out["db3"] = list(dU.sum(0).to(dt).split(widths))
    return out


# ------------------------------------------------------------------ one pass

def _own(s, case):
    tp = s["tp"]
    if case["op"] == "qk_fwd":
        return s["proj"].qk_norm_rope_forward(s["QKV"], positions=s["pos"], gq=s["gq"], gk=s["gk"])
    if case["op"] == "qk_bwd":
        dQKV, dgq, dgk = s["proj"].qk_norm_rope_backward(s["QKV"], s["dQK"], positions=s["pos"], gq=s["gq"],
                                                         gk=s["gk"], dV_i=s["dV"])
        return {"dQKV": dQKV, "dgq": dgq, "dgk": dgk}
    if case["op"] == "keep":
        return tp.ckpt8_unpack(tp.ckpt8_pack(s["x"]), case["T"], case["w"], case["dtype"])
    mlp, out = s["mlp"], {}
    if case["op"] == "mlp_step":
        out["Y"], ckpt = mlp.forward_ckpt8(s["X"], s["W1"], s["W2"], s["W3"], b1_i=s["b1"], b3_i=s["b3"], b2=s["b2"])
    else:
        ckpt = s["ckpt"]
    g = mlp.backward_ckpt8(s["X"], s["W1"], s["W2"], ckpt, s["dY"], s["W3"], bias_grads=case["bias"])
    names = ["dX", "dW1", "dW2"] + (["dW3"] if case["act"] == "swiglu" else [])
    names += (["db1", "db2"] + (["db3"] if case["act"] == "swiglu" else [])) if case["bias"] else []
    return out | {n: g[n] for n in names}


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "qk_fwd":
        return _plain_qk_fwd(state, case)
    if case["op"] == "qk_bwd":
        return _plain_qk_bwd(state, case)
    if case["op"] == "keep":
        return _values(*_quantise(state["x"].float()), case["w"]).to(DTYPES[case["dtype"]])
    return _plain_mlp(state, case)


def work(case):
    es, T = (2 if case["dtype"] == "bf16" else 4), case["T"]
    if case["op"] in ("qk_fwd", "qk_bwd"):
        qk, v, D = sum(_w(case["dq"])) + sum(_w(case["dkv"])), sum(_w(case["dkv"])), case["D"]
        if case["op"] == "qk_fwd":  # q and k in and out, gains, positions
            return {"bytes": es * (2 * T * qk + 2 * D) + 8 * T, "flops": 9 * T * qk}
        return {"bytes": es * (3 * T * qk + 2 * T * v + 4 * D) + 8 * T, "flops": 18 * T * qk}
    if case["op"] == "keep":  # the tensor in, its checkpoint out and in, the tensor out
        kept = 544 * -(-T // 32) * -(-case["w"] // 16)
        return {"bytes": 2 * es * T * case["w"] + 2 * kept, "flops": 4 * T * case["w"]}
    widths, d, sw = _w(case["widths"]), case["d"], case["act"] == "swiglu"
    dff, n = sum(widths), (2 if sw else 1)
    kept = sum(544 * -(-T // 32) * -(-w // 16) for w in widths * n)
    step = case["op"] == "mlp_step"
    acts = 4 if step else 3  # X, dY, dX, and Y of the forward pass
    bias = es * 2 * (n * dff + d) if case["bias"] else 0
    return {"bytes": es * (acts * T * d + 2 * (n + 1) * d * dff) + (2 if step else 1) * kept + bias,
            "flops": (2 * (n + 1) * (3 if step else 2)) * T * d * dff}


# ------------------------------------------------------------------ 64 bits, from the definitions

def _keep64(x):
    rows, cols = x.shape
    G = -(-cols // 16)
    p = torch.zeros(rows, G * 16, dtype=torch.float64, device=x.device)
    p[:, :cols] = x
    p = p.view(rows, G, 16)
    m = p.abs().max(-1, keepdim=True).values
    # the smallest e with m <= 448 * 2^e
    e = torch.ceil(torch.log2(torch.where(m > 0, m, torch.ones_like(m)) / 448.0))
    e = torch.where(448.0 * torch.exp2(e - 1) >= m, e - 1, e)
    e = torch.where(448.0 * torch.exp2(e) < m, e + 1, e)
    e = torch.where(m > 0, e, torch.full_like(e, -117.0)).clamp(-117.0, 120.0)
    v = p / torch.exp2(e)
    # e4m3: 3 bits behind the leading one, multiples of 2^-9 below 2^-6
    mag = v.abs()
    low = torch.floor(torch.log2(mag.clamp_min(2.0 ** -6)))
    low = torch.where(torch.exp2(low) > mag.clamp_min(2.0 ** -6), low - 1, low)
    low = torch.where(torch.exp2(low + 1) <= mag, low + 1, low)
    step = torch.exp2(low - 3)
    return ((v / step).round() * step * torch.exp2(e)).view(rows, G * 16)[:, :cols]


def _decode64(buf, rows, cols):
    """The values of a stored checkpoint, from the bits of its codes."""
    G = -(-cols // 16)
    r = torch.arange(rows, device=buf.device)[:, None]
    c = torch.arange(cols, device=buf.device)[None]
    block = (r // 32) * G + c // 16
    code = buf[block * 512 + (r % 32) * 16 + c % 16].long()
    scale = buf[-(-rows // 32) * G * 512 + block * 32 + r % 32].double() - 127
    ex, man = (code >> 3) & 15, (code & 7).double()
    v = torch.where(ex > 0, (1 + man / 8) * torch.exp2(ex.double() - 7), man / 512)
    return torch.where(code >= 128, -v, v) * torch.exp2(scale)


def _exact_qk(s, case):
    dq, dkv, D, R = _w(case["dq"]), _w(case["dkv"]), case["D"], case["R"]
    j = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    ang = s["pos"].double().view(-1, 1, 1) * torch.exp(-2 * j / max(R, 1) * math.log(10000.0))
    turn = torch.complex(ang.cos(), ang.sin())
    ia, ib = (torch.arange(R // 2), torch.arange(R // 2) + R // 2) if case["layout"] == "halves" else \
        (2 * torch.arange(R // 2), 2 * torch.arange(R // 2) + 1)
    ia, ib = ia.cuda(), ib.cuda()

    def spin(x, by):
        z = torch.complex(x[..., ia], x[..., ib]) * by
        y = x.clone()
        y[..., ia], y[..., ib] = z.real, z.imag
        return y

    fwd, outs, dgs = case["op"] == "qk_fwd", [], [torch.zeros(D, dtype=torch.float64, device="cuda") for _ in "qk"]
    for i, x in enumerate(s["QKV"]):
        parts = []
        for kind, (o, w, g) in enumerate(((0, dq[i], s["gq"]), (dq[i], dkv[i], s["gk"]))):
            h = x[:, o:o + w].double().view(case["T"], -1, D)
            rms = (h.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt()
            if fwd:
                parts.append(spin(h / rms * g.double(), turn).flatten(1))
                continue
            dy = spin(s["dQK"][i][:, o:o + w].double().view(case["T"], -1, D), turn.conj())
            dgs[kind] += (dy * h / rms).sum((0, 1))
            dn = dy * g.double()
            parts.append((dn / rms - h * (dn * h).sum(-1, keepdim=True) / (D * rms.pow(3))).flatten(1))
        if not fwd:
            parts.append(s["dV"][i].double())
        outs.append(torch.cat(parts, 1))
    return outs if fwd else {"dQKV": outs, "dgq": dgs[0], "dgk": dgs[1]}


def _exact_mlp(s, case):
    sw, step, T = case["act"] == "swiglu", case["op"] == "mlp_step", case["T"]
    X, dY, n = s["X"].double(), s["dY"].double(), len(s["W1"])
    Y, dX = torch.zeros_like(X), torch.zeros_like(X)
    out = {"dW1": [], "dW2": [], "dW3": [], "db1": [], "db3": []}
    for i in range(n):
        W1, W2 = s["W1"][i].double(), s["W2"][i].double()
        W3 = s["W3"][i].double() if sw else None
        U = None
        if step:
            A = X @ W1 + (s["b1"][i].double() if s["b1"] else 0)
            if sw:
                U = X @ W3 + (s["b3"][i].double() if s["b3"] else 0)
            Y += (U * A / (1 + torch.exp(-A)) if sw else 0.5 * A * torch.erfc(-A / math.sqrt(2))) @ W2
            A, U = _keep64(A), _keep64(U) if sw else None
        else:
            A = _decode64(s["ckpt"][i], T, W1.shape[1])
            U = _decode64(s["ckpt"][n + i], T, W1.shape[1]) if sw else None
        dH = dY @ W2.T
        if sw:
            sg = 1 / (1 + torch.exp(-A))
            H, dU = U * A * sg, dH * A * sg
            dA = dH * U * sg * (1 + A * (1 - sg))
            out["dW3"].append(X.T @ dU)
            out["db3"].append(dU.sum(0))
            dX += dU @ W3.T
        else:
            cdf = 0.5 * torch.erfc(-A / math.sqrt(2))
            H, dA = A * cdf, dH * (cdf + A * torch.exp(-A * A / 2) / math.sqrt(2 * math.pi))
        out["dW2"].append(H.T @ dY)
        out["dW1"].append(X.T @ dA)
        out["db1"].append(dA.sum(0))
        dX += dA @ W1.T
    out["dX"] = dX
    if step:
        out["Y"] = Y + (s["b2"].double() if s["b2"] is not None else 0)
    if case["bias"]:
        out["db2"] = dY.sum(0)
    drop = ([] if sw else ["dW3", "db3"]) + ([] if case["bias"] else ["db1", "db3"])
    return {k: v for k, v in out.items() if k not in drop}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("qk_fwd", "qk_bwd"):
        return _exact_qk(s, case)
    if case["op"] == "keep":
        return _keep64(s["x"].double())
    return _exact_mlp(s, case)
