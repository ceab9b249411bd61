"""Cases for measuring what a training step needs around the block's GEMM launches.

norm_fwd, norm_bwd  layer norm or RMS norm of the tokens in front of a block, with the residual stream's sum; its
                    backward pass with the gradients of gain and bias (tpmlp_norm_forward, tpmlp_norm_backward)
proj, row           the two row-parallel products with the residual stream added in the epilogue: the attention
                    block's output projection and the MLP's second product (tpmlp_attn_out_forward_residual,
                    tpmlp_forward_row_residual)
adamw               an AdamW step over all tensors, moments in 32 or 8 bits, with the gradients' global norm clipped
                    (tpmlp_grad_norm, tpmlp_adamw_step); moments in 8 bits are read out as well, as they are when a
                    state is looked at (tpmlp_adamw8_unpack)

`own` chooses between the plain form (elementary torch operations in 32 bits) and the library's kernels.

Moments in 8 bits, of a tensor of n elements: groups of 256, the last one filled up with zeros.  M a group's largest
magnitude, e = floor(log2 M), one more where M > 1.875 * 2^e; at least -90.  A magnitude is kept as a code c of 7 bits
(first moment, its sign in bit 7; S = 15) or 8 bits (second; S = 31), which stands for (1 + (c % 8) / 8) * 2^(c // 8)
* 2^(e - S), c = 0 for 0.  Rounding is stochastic: with r in [0, 2^16) the two neighbours' upper one is taken where
the distance from the lower, over the gap, is at least 1 - r / 2^16; below the smallest code (x = y * 2^(e - S), y <
1.125) the first moment is kept as that code where 2^16 y > 1.125 r, else as 0, and a second moment above 0 as that code.
r of element i of tensor k: with h(x) an integer hash of 32 bits, key = h(h(h(h(seed low) ^ seed high) ^ step low) ^
step high), group number q counted over all tensors' groups, a = h(h(key ^ q low) ^ q high), l = i % 256: the low half
of h(a + (l // 2) * 0x9E3779B9) for even l, the high half for odd l.  Storage: the groups' codes, 256 bytes each, then a
byte e + 91 per group (0: all zero).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
G = 256  # elements of a group
HYPER = {"lr": 3e-4, "betas": (0.9, 0.999), "eps": 1e-8}
DECAY = 0.1  # of the matrices; vectors (gains, biases) have none


def _w(text):
    return [int(v) for v in text.split(",")]


def listed():
    c3 = "3145728,5242880,4194304,4194304"  # W1 and W2 of the GeLU block of 2048, shards of 1536, 2560, 2048, 2048
    half = ",".join(["22544384"] * 6)  # W1, W3, W2 of the SwiGLU block of 4096, two shards of 5504
    odd = "69696,264,264,264,19008,52800,35904,72,200,136,72,200,136,19008,52800,35904,1,7,513,65793"
    return [
        # one new token of a model of 4096; latency counts
        {"name": "norm_fwd token", "op": "norm_fwd", "T": 1, "d": 4096, "kind": "rms", "bias": False, "add": False,
         "dtype": "bf16"},
        # the tokens in front of the SwiGLU block, the sublayer's output added to the residual stream on the way
        {"name": "norm_fwd batch", "op": "norm_fwd", "T": 8192, "d": 4096, "kind": "rms", "bias": False, "add": True,
         "dtype": "bf16"},
        # an odd number of tokens, a width that fills no whole round of threads, fp32
        {"name": "norm_fwd ragged", "op": "norm_fwd", "T": 1533, "d": 264, "kind": "layer", "bias": True, "add": True,
         "dtype": "fp32"},
        # the widest hidden size of the attention projections' workloads, with the residual stream's own gradient
        {"name": "norm_bwd wide", "op": "norm_bwd", "T": 8192, "d": 16384, "kind": "rms", "bias": False, "add": True,
         "dtype": "bf16"},
        # the GPT-2-small block
        {"name": "norm_bwd small", "op": "norm_bwd", "T": 8192, "d": 768, "kind": "layer", "bias": True, "add": True,
         "dtype": "bf16"},
        # few odd tokens, fp32
        {"name": "norm_bwd ragged", "op": "norm_bwd", "T": 777, "d": 2048, "kind": "layer", "bias": True, "add": False,
         "dtype": "fp32"},
        # the output projection of 8 shards of four heads of 128
        {"name": "proj batch", "op": "proj", "T": 8192, "d": 4096, "widths": ",".join(["512"] * 8), "bias": False,
         "dtype": "bf16"},
        # the GPT-2-small block's second product, 4 shards, with its bias
        {"name": "row small", "op": "row", "T": 8192, "d": 768, "widths": "768,768,768,768", "bias": True,
         "dtype": "bf16"},
        # a short batch, unequal shards whose widths fill no tile, fp32
        {"name": "row ragged", "op": "row", "T": 203, "d": 264, "widths": "72,200,136", "bias": True, "dtype": "fp32"},
        # gains, biases and matrices of a small ragged model, 8-bit moments
        {"name": "adamw ragged", "op": "adamw", "sizes": odd, "dtype": "bf16", "grads": "bf16", "bits": 8,
         "master": False, "clip": True},
        # the GeLU block of 2048: bf16 weights with fp32 masters, moments in 32 bits
        {"name": "adamw master", "op": "adamw", "sizes": c3 + "," + c3, "dtype": "bf16", "grads": "bf16", "bits": 32,
         "master": True, "clip": True},
        # the SwiGLU block of 4096 with 8-bit moments
        {"name": "adamw 8 bits", "op": "adamw", "sizes": half, "dtype": "bf16", "grads": "bf16", "bits": 8,
         "master": False, "clip": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "proj", "row", "adamw", "adamw"])
    if op in ("norm_fwd", "norm_bwd"):
        d, kind = 8 * _log(rng, 4, 2048), rng.choice(["layer", "rms"])
        return {"op": op, "T": _log(rng, 1, min(16384, 8192 * 8192 // d)), "d": d, "kind": kind,
                "bias": kind == "layer", "add": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op in ("proj", "row"):
        small = rng.random() < 0.3  # fp32 storage: small blocks
        t = rng.randint(1, 4 if small else 8)
        return {"op": op, "T": _log(rng, 1, 256 if small else 8192),
                "d": 4 * rng.randint(8, 64) if small else 8 * _log(rng, 8, 512),
                "widths": ",".join(str(4 * rng.randint(4, 64) if small else 8 * _log(rng, 8, 64)) for _ in range(t)),
                "bias": op == "row" and rng.random() < 0.5, "dtype": "fp32" if small else "bf16"}
    sizes = [_log(rng, 1, 1 << 23) for _ in range(rng.randint(1, 15))]
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    return {"op": op, "sizes": ",".join(map(str, sizes)), "dtype": dtype,
            "grads": "fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"]), "bits": rng.choice([8, 32]),
            "master": dtype == "bf16" and rng.random() < 0.5, "clip": rng.random() < 0.7}


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def normal(*shape, std=1.0):
        return (randn(*shape) * std).to(dt)

    if case["op"] in ("norm_fwd", "norm_bwd"):
        T, d = case["T"], case["d"]
        # a residual stream: some columns much larger than the others and off zero, tokens of different sizes
        col = torch.exp(0.5 * randn(d))
        s = {"x": (randn(T, d) * col * torch.exp(0.3 * randn(T, 1)) + 0.3 * randn(d)).to(dt),
             "gain": (1 + 0.1 * randn(d)).to(dt), "b": (0.1 * randn(d)).to(dt) if case["bias"] else None}
        if case["op"] == "norm_fwd":
            s["r"] = normal(T, d) if case["add"] else None
        else:
            s["dy"] = normal(T, d)
            s["dsum"] = normal(T, d) if case["add"] else None
            x = s["x"].double()
            mu = x.mean(1) if case["kind"] == "layer" else torch.zeros(T, dtype=torch.float64, device="cuda")
            var = (x - mu[:, None]).square().mean(1)
            s["stats"] = torch.stack([mu, (var + EPS).rsqrt()], 1).float()
        return s
    if case["op"] in ("proj", "row"):
        T, d, widths = case["T"], case["d"], _w(case["widths"])
        return {"H": [normal(T, w) for w in widths], "W": [normal(w, d, std=0.02) for w in widths], "R": normal(T, d),
                "b2": normal(d, std=0.1) if case["bias"] else None}
    sizes, gd = _w(case["sizes"]), DTYPES[case["grads"]]
    s = {"g": [], "p": [], "master": [] if case["master"] else None, "m": [], "v": [], "sizes": sizes,
         "rng": int(torch.randint(0, 1 << 62, (1,), generator=gen, device="cuda"))}
    for n in sizes:  # gradients of different sizes, a part of them exactly zero
        size = 1e-3 * torch.exp(randn(-(-n // 64)).repeat_interleave(64)[:n])
        g = randn(n) * size
        g[: n // 16] = 0
        w = 0.02 * randn(n)
        s["g"].append(g.to(gd))
        s["p"].append(w.to(dt))
        if case["master"]:
            s["master"].append(w)
        m, v = 0.5 * randn(n) * size, size.square() * torch.exp(0.5 * randn(n))
        m[: n // 32] = 0
        v[: n // 32] = 0
        if case["bits"] == 8:  # from an earlier step
            m, v = (_bytes(x, k) for x, k in ((m, 0), (v, 1)))
        s["m"].append(m)
        s["v"].append(v)
    s["steps"] = 400  # done so far
    return s


def _max_norm(case):
    """Clips: the gradients' norm is about 2.7e-3 times the root of their number."""
    return 1e-3 * math.sqrt(sum(_w(case["sizes"]))) if case["clip"] else None


def _decays(case):
    return [DECAY if n >= 4096 else 0.0 for n in _w(case["sizes"])]


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "adamw":
        s["of"] = torch.tensor(s["sizes"], device="cuda")
        s["decay"] = torch.tensor(_decays(case), device="cuda")
    if own:  # the plan, its workspace and the optimizer, which a program keeps
        import megatron_tensor_transformer_column_gb300 as tp

        if case["op"] in ("norm_fwd", "norm_bwd"):
            s["norm"] = tp.TokenNorm(case["T"], case["d"], case["kind"], case["dtype"], eps=EPS)
        elif case["op"] == "proj":
            widths = _w(case["widths"])
            s["proj"] = tp.ShardedAttentionProj(case["T"], case["d"], widths, widths, case["dtype"])
        elif case["op"] == "row":
            s["mlp"] = tp.ShardedMLP(case["T"], case["d"], _w(case["widths"]), "gelu", case["dtype"])
        else:
            s["opt"] = tp.ShardedAdamW(s["p"], **HYPER, weight_decay=_decays(case), bits=case["bits"],
                                       master=s["master"], max_norm=_max_norm(case), seed=s["rng"])
            s["opt"].load_moments(s["m"], s["v"], steps=s["steps"])
    return s


# ------------------------------------------------------------------ moments in 8 bits, plain form

def _bits(x):
    return x.contiguous().view(torch.int32)


def _encode(x, second, r):
    """[groups x 256] fp32 and r -> (codes, e)."""
    S = 31 if second else 15
    a = x.abs()
    big = _bits(a.amax(-1))
    e = torch.where(big > 0, ((big + 0xFFFFF) >> 23) - 127, torch.full_like(big, -91)).clamp_min(-90)
    w = _bits(a) - ((e + 127 - S) << 23)[:, None]
    c = (w + (r << 4)) >> 20
    if second:
        low = (a > 0).int()
    else:
        low = (torch.ldexp(a, (S - e)[:, None]) * 65536 > r.float() * 1.125).int()
    c = torch.where(w < 1 << 20, low, c)
    if not second:
        c = torch.where(x < 0, c + 128, c)
    zero = big == 0
    return torch.where(zero[:, None], 0, c).to(torch.uint8), torch.where(zero, -91, e)


def _decode(codes, e, second):
    S = 31 if second else 15
    c = codes.int()
    mag = c if second else c & 127
    v = ((mag << 20) + ((e + 127 - S) << 23)[:, None]).view(torch.float32)
    v = torch.where(mag == 0, 0.0, v)
    return v if second else torch.where(c > 127, -v, v)


def _bytes(x, second):
    """A moment as it lies in memory, rounded to the nearest code."""
    n = x.numel()
    x = torch.nn.functional.pad(x, (0, -n % G)).view(-1, G)
    c, e = _encode(x, second, torch.full_like(x, 1 << 15, dtype=torch.int32))
    return torch.cat([c.view(-1), (e + 91).to(torch.uint8)])


def _groups(bufs, sizes):
    """The tensors' codes and scales side by side."""
    groups = [-(-n // G) for n in sizes]
    c = torch.cat([b[: k * G] for b, k in zip(bufs, groups)]).view(-1, G)
    return c, torch.cat([b[k * G:] for b, k in zip(bufs, groups)]).int() - 91


def _hash(x):
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(seed, step, groups):
    """r of every element of the groups."""
    key = 0
    for part in (seed & 0xFFFFFFFF, seed >> 32, step & 0xFFFFFFFF, step >> 32):
        key = _hash(key ^ part)
    q = torch.arange(groups, device="cuda")
    a = _hash(_hash(key ^ (q & 0xFFFFFFFF)) ^ (q >> 32))
    h = _hash((a[:, None] + torch.arange(G // 2, device="cuda") * 0x9E3779B9) & 0xFFFFFFFF)
    return torch.stack([h & 0xFFFF, h >> 16], -1).flatten(1).int()


# ------------------------------------------------------------------ plain forms

def _plain_norm_fwd(s, case):
    x = s["x"].float()
    out = {}
    if s["r"] is not None:  # the sum is kept in the storage type, and what is kept is normed
        out["sum"] = (x + s["r"].float()).to(s["x"].dtype)
        x = out["sum"].float()
    mu = x.mean(1, keepdim=True) if case["kind"] == "layer" else x.new_zeros(x.shape[0], 1)
    c = x - mu
    r = torch.rsqrt(c.square().mean(1, keepdim=True) + EPS)
    y = c * r * s["gain"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    return out | {"y": y.to(s["x"].dtype), "stats": torch.cat([mu, r], 1)}


def _plain_norm_bwd(s, case):
    dt, dy, (mu, r) = s["x"].dtype, s["dy"].float(), s["stats"].split(1, 1)
    n = (s["x"].float() - mu) * r
    w = dy * s["gain"].float()
    dx = w - n * (w * n).mean(1, keepdim=True)
    if case["kind"] == "layer":
        dx = dx - w.mean(1, keepdim=True)
    dx = dx * r
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    out = {"dx": dx.to(dt), "dgain": (dy * n).sum(0).to(dt)}
    return out | ({"dbias": dy.sum(0).to(dt)} if case["bias"] else {})


def _plain_product(s):
    y = torch.cat(s["H"], 1).float() @ torch.cat(s["W"], 0).float() + s["R"].float()
    return (y if s["b2"] is None else y + s["b2"].float()).to(s["R"].dtype)


def _plain_adamw(s, case):
    sizes, lr, (b1, b2) = s["sizes"], HYPER["lr"], HYPER["betas"]
    s["steps"] += 1
    t, out = s["steps"], {}
    g = torch.cat(s["g"]).float()
    if case["clip"]:
        out["norm"] = g.double().square().sum().sqrt().float()
        most = _max_norm(case)
        g = g * torch.where(out["norm"] > most, most / out["norm"], 1.0)
    p = torch.cat(s["master"] or s["p"]).float()
    if case["bits"] == 8:
        pad = [-n % G for n in sizes]
        at = torch.cat([s["of"].new_ones(n + k).cumsum(0) <= n for n, k in zip(sizes, pad)])

        def back(x):  # without what fills up the last groups
            return x.view(-1)[at]

        (mc, me), (vc, ve) = _groups(s["m"], sizes), _groups(s["v"], sizes)
        m, v = back(_decode(mc, me, False)), back(_decode(vc, ve, True))
    else:
        m, v = torch.cat(s["m"]), torch.cat(s["v"])
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * (1 - b2) * g
    den = v.sqrt() * (1 / math.sqrt(1 - b2 ** t)) + HYPER["eps"]
    wd = torch.repeat_interleave(s["decay"], s["of"])
    p = p - p * (lr * wd) - (lr / (1 - b1 ** t)) * m / den
    for dst, src in zip(s["master"] or s["p"], p.split(sizes)):
        dst.copy_(src)
    if case["master"]:
        out["master"] = s["master"]
        for dst, src in zip(s["p"], s["master"]):
            dst.copy_(src)
    out["p"] = s["p"]
    if case["bits"] == 32:
        for dst, src in zip(s["m"] + s["v"], m.split(sizes) + v.split(sizes)):
            dst.copy_(src)
        return out | {"m": s["m"], "v": s["v"]}
    r = _random(s["rng"], t, at.numel() // G)
    for name, x, second in (("m", m, False), ("v", v, True)):
        full = x.new_zeros(at.numel())
        full[at] = x
        c, e = _encode(full.view(-1, G), second, r)
        groups = [(n + k) // G for n, k in zip(sizes, pad)]
        for buf, cs, es, k in zip(s[name], c.split(groups), e.split(groups), groups):
            buf[: k * G].copy_(cs.view(-1))
            buf[k * G:].copy_(es + 91)
        out[name] = list(back(_decode(c, e, second)).bfloat16().split(sizes))
    return out


# ------------------------------------------------------------------ one pass

def _own(s, case):
    if case["op"] == "norm_fwd":
        y, stats, total = s["norm"].forward(s["x"], s["gain"], s["b"], residual=s["r"])
        return {"y": y, "stats": stats} | ({"sum": total} if case["add"] else {})
    if case["op"] == "norm_bwd":
        dx, dgain, dbias = s["norm"].backward(s["x"], s["stats"], s["dy"], s["gain"], dsum=s["dsum"],
                                              bias_grad=case["bias"])
        return {"dx": dx, "dgain": dgain} | ({"dbias": dbias} if case["bias"] else {})
    if case["op"] == "proj":
        return s["proj"].out_forward(s["W"], s["H"], residual=s["R"])
    if case["op"] == "row":
        return s["mlp"].row_forward(s["H"], s["W"], b2=s["b2"], residual=s["R"])
    opt, out = s["opt"], {}
    norm = opt.step(s["g"])
    if case["clip"]:
        out["norm"] = norm
    if case["master"]:
        out["master"] = s["master"]
    m, v = opt.moments()
    return out | {"p": s["p"], "m": m, "v": v}


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "norm_fwd":
        return _plain_norm_fwd(state, case)
    if case["op"] == "norm_bwd":
        return _plain_norm_bwd(state, case)
    if case["op"] in ("proj", "row"):
        return _plain_product(state)
    return _plain_adamw(state, case)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm_fwd", "norm_bwd"):
        n, d = case["T"] * case["d"], case["d"]
        arrays = (4 if case["add"] else 2) if case["op"] == "norm_fwd" else (4 if case["add"] else 3)
        vectors = (2 if case["bias"] else 1) if case["op"] == "norm_fwd" else (3 if case["bias"] else 2)
        return {"bytes": es * (arrays * n + vectors * d) + 8 * case["T"],
                "flops": (9 if case["op"] == "norm_fwd" else 15) * n}
    if case["op"] in ("proj", "row"):
        T, d, k = case["T"], case["d"], sum(_w(case["widths"]))
        return {"bytes": es * (T * k + k * d + 2 * T * d + (d if case["bias"] else 0)), "flops": 2 * T * d * k}
    n, gs = sum(_w(case["sizes"])), 2 if case["grads"] == "bf16" else 4
    weights = es + 8 if case["master"] else 2 * es  # bf16 weights with a master are written only
    # moments in and out; in 8 bits also the 2 bytes each that they are read out as
    moments = 16 if case["bits"] == 32 else 2 * (2 + 2 / G) + 4
    return {"bytes": n * (gs + weights + moments), "flops": 20 * n}


# ------------------------------------------------------------------ 64 bits, from the definitions

def _exact_norm(s, case):
    x = s["x"].double()
    out = {}
    if case["op"] == "norm_fwd":
        if s["r"] is not None:
            total = x + s["r"].double()
            out["sum"] = total
            x = total.to(s["x"].dtype).double()  # kept in the storage type
        var, mu = torch.var_mean(x, 1, correction=0, keepdim=True)
        if case["kind"] == "rms":
            var, mu = x.pow(2).sum(1, keepdim=True) / case["d"], torch.zeros_like(mu)
        std = (var + EPS).sqrt()
        out["y"] = (x - mu) / std * s["gain"].double() + (s["b"].double() if s["b"] is not None else 0)
        out["stats"] = torch.cat([mu, 1 / std], 1)
        return out
    mu, r, dy = s["stats"][:, :1].double(), s["stats"][:, 1:].double(), s["dy"].double()
    n = (x - mu) * r
    w = dy * s["gain"].double()
    # the gradient of the norm along n, and along the ones where the mean is taken away
    dx = w - n * torch.einsum("ij,ij->i", w, n)[:, None] / case["d"]
    if case["kind"] == "layer":
        dx -= w.sum(1, keepdim=True) / case["d"]
    dx *= r
    if s["dsum"] is not None:
        dx += s["dsum"].double()
    out = {"dx": dx, "dgain": torch.einsum("ij,ij->j", dy, n)}
    return out | ({"dbias": torch.einsum("ij->j", dy)} if case["bias"] else {})


def _round64(x, second, r):
    """Values that the 8-bit form of x [groups x 256] stands for, from its definition."""
    S = 31 if second else 15
    a = x.abs()
    most = a.max(1, keepdim=True).values
    man, ex = torch.frexp(most)  # most = man 2^ex, man in [0.5, 1)
    e = (ex - 1 + (man > 0.9375).int()).clamp_min(-90)
    man, ex = torch.frexp(a)
    eighths = man * 16  # [8, 16)
    low = torch.floor(eighths)
    up = (eighths - low >= 1 - r.double() / 65536).double()
    kept = torch.ldexp((low + up) / 8, ex - 1)
    least = torch.ldexp(torch.ones_like(most), e - S)
    take = a > 0 if second else a * 65536 > least * 1.125 * r.double()
    kept = torch.where(a < 1.125 * least, torch.where(take, 1.125 * least, torch.zeros_like(a)), kept)
    return torch.where(most > 0, torch.where(x < 0, -kept, kept), torch.zeros_like(a))


def _values64(buf, n, second):
    """The values of a stored moment, from the bits of its codes."""
    i = torch.arange(n, device=buf.device)
    groups = -(-n // G)
    code, scale = buf[i].long(), buf[groups * G + i // G].double() - 91
    mag = code if second else code % 128
    v = (1 + (mag % 8).double() / 8) * torch.exp2(torch.div(mag, 8, rounding_mode="floor") + scale - (31 if second else 15))
    v = torch.where(mag == 0, torch.zeros_like(v), v)
    return v if second else torch.where(code >= 128, -v, v)


def _random64(seed, step, first, groups, device):
    """r of every element of the groups first, first + 1, ..., in steps of 32 bits."""
    mask = (1 << 32) - 1

    def mix(x):
        x = x ^ (x >> 16)
        x = (x * 0x7FEB352D) & mask
        x = x ^ (x >> 15)
        x = (x * 0x846CA68B) & mask
        return x ^ (x >> 16)

    key = mix(mix(mix(mix(seed & mask) ^ (seed >> 32)) ^ (step & mask)) ^ (step >> 32))
    q = torch.arange(first, first + groups, device=device, dtype=torch.int64)[:, None]
    pair = torch.arange(G, device=device, dtype=torch.int64)[None] // 2
    h = mix((mix(mix((q & mask) ^ key) ^ (q >> 32)) + pair * 0x9E3779B9) & mask)
    odd = torch.arange(G, device=device)[None] % 2 == 1
    return torch.where(odd, h >> 16, h & 0xFFFF)


def _exact_adamw(s, case):
    lr, (b1, b2), t = HYPER["lr"], HYPER["betas"], s["steps"] + 1
    f, out = 1.0, {"p": [], "m": [], "v": []}
    if case["clip"]:
        out["norm"] = torch.stack([g.double().pow(2).sum() for g in s["g"]]).sum().sqrt()
        f = min(1.0, _max_norm(case) / float(out["norm"]))
    first = 0
    for k, n in enumerate(s["sizes"]):
        g = s["g"][k].double() * f
        p = (s["master"] or s["p"])[k].double()
        m, v = s["m"][k], s["v"][k]
        if case["bits"] == 8:
            m, v = _values64(m, n, False), _values64(v, n, True)
        m = b1 * m.double() + (1 - b1) * g
        v = b2 * v.double() + (1 - b2) * g * g
        step = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + HYPER["eps"])
        out["p"].append(p - lr * (step + _decays(case)[k] * p))
        if case["bits"] == 8:
            groups = -(-n // G)
            r = _random64(s["rng"], t, first, groups, g.device)
            m, v = (_round64(torch.nn.functional.pad(x, (0, -n % G)).view(-1, G), second, r).view(-1)[:n]
                    for x, second in ((m, False), (v, True)))
            first += groups
        out["m"].append(m)
        out["v"].append(v)
    if case["master"]:
        out["master"] = out["p"]
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        return _exact_norm(s, case)
    if case["op"] in ("proj", "row"):
        y = s["R"].double() + (s["b2"].double() if s["b2"] is not None else 0)
        for h, w in zip(s["H"], s["W"]):
            y = y + h.double() @ w.double()
        return y
    return _exact_adamw(s, case)
