"""The head norm with rotation and the 8-bit checkpoints together, as a layer's training step uses them between the
library's GEMM launches: QKV projection, norm and rotation, an attention core (plain torch here), output projection,
MLP block, and all of it backward from what was kept in 8 bits (QKV by pack, the pre-activations by the block).

The reference runs the same formulas in 64 bits; its backward pass takes the kept values, read back from the device.
Tolerance: at most ten tensors rounded to bf16 lie between an input and any result, each off by 2^-8 of its value:
10 * 2^-8 of the largest reference value."""
import numpy as np
import pytest
import torch

import operators_reference as ref

pytestmark = pytest.mark.gpu

T, d, D = 160, 128, 64
DQ, DKV = [128, 64], [64, 64]
WIDTHS = [192, 72]
TOL = 10 * 2.0 ** -8


def core(q, k, v, mask):
    """Causal attention of [T, H, D] heads (grouped keys), elementary operations."""
    g = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("thd,shd->hts", q, k) / D ** 0.5
    p = torch.softmax(s.masked_fill(~mask, float("-inf")), -1)
    return torch.einsum("hts,shd->thd", p, v)


def core_of_shard(QK, V, i, mask):
    x = QK[i]
    split = lambda t: t.reshape(T, -1, D)
    return core(split(x[:, :DQ[i]]), split(x[:, DQ[i]:]), split(V[i]), mask).reshape(T, -1)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_layer_step(gpu_lib, act):
    tp = gpu_lib
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(torch.bfloat16).cuda()
    X, dY = rnd(T, d), rnd(T, d)
    Wqkv = [rnd(d, q + 2 * k, std=0.1) for q, k in zip(DQ, DKV)]
    WO = [rnd(q, d, std=0.1) for q in DQ]
    W1, W2 = [rnd(d, w, std=0.1) for w in WIDTHS], [rnd(w, d, std=0.1) for w in WIDTHS]
    W3 = [rnd(d, w, std=0.1) for w in WIDTHS] if act == "swiglu" else None
    gq, gk = 1 + rnd(D, std=0.1), 1 + rnd(D, std=0.1)
    pos = torch.cat([torch.arange(96), torch.arange(T - 96)]).cuda()  # two sequences behind one another
    seq = torch.cat([torch.zeros(96), torch.ones(T - 96)]).cuda()
    mask = (seq[:, None] == seq[None]) & (pos[:, None] >= pos[None])

    proj = tp.ShardedAttentionProj(T, d, DQ, DKV, "bf16")
    proj.set_qk_norm_rope(D)
    mlp = tp.ShardedMLP(T, d, WIDTHS, act, "bf16")

    # forward; what is kept: X, X2, QKV in 8 bits, O, the core's inputs, the block's checkpoints
    QKV = proj.qkv_forward(X, Wqkv)
    kept = [tp.ckpt8_pack(x) for x in QKV]
    QK = [x.float().requires_grad_() for x in proj.qk_norm_rope_forward(QKV, pos, gq, gk)]
    V = [x[:, q + k:].float().requires_grad_() for x, q, k in zip(QKV, DQ, DKV)]
    O32 = [core_of_shard(QK, V, i, mask) for i in range(2)]
    O = [o.detach().bfloat16() for o in O32]
    X2 = X + proj.out_forward(WO, O)
    Y, ckpt = mlp.forward_ckpt8(X2, W1, W2, W3)

    # backward
    g = mlp.backward_ckpt8(X2, W1, W2, ckpt, dY, W3)
    dO, dWO = proj.out_backward(WO, O, g["dX"])
    torch.autograd.backward(O32, [x.float() for x in dO])
    x8 = [tp.ckpt8_unpack(c, T, q + 2 * k) for c, q, k in zip(kept, DQ, DKV)]
    dQKV, dgq, dgk = proj.qk_norm_rope_backward(x8, [x.grad.bfloat16() for x in QK], pos, gq, gk,
                                                dV_i=[v.grad.bfloat16() for v in V])
    dX, dWqkv = proj.qkv_backward(X, Wqkv, dQKV)
    dX = dX + g["dX"]
    torch.cuda.synchronize()
    proj.check()
    mlp.check()

    # the same in 64 bits
    c = lambda x: x.detach().double().cpu()
    freq, p = ref.frequencies(D), pos.cpu().numpy()
    X64, m = c(X), mask.cpu()
    QKV64 = [X64 @ c(w) for w in Wqkv]
    heads = lambda x: x.numpy().reshape(T, -1, D)
    QK64, V64 = [], []
    for x, q, k in zip(QKV64, DQ, DKV):
        yq = ref.heads_forward(heads(x[:, :q]), p, freq, "halves", c(gq).numpy(), 1e-6)[0]
        yk = ref.heads_forward(heads(x[:, q:q + k]), p, freq, "halves", c(gk).numpy(), 1e-6)[0]
        QK64.append(torch.from_numpy(np.concatenate([yq, yk], 1).reshape(T, -1)).requires_grad_())
        V64.append(x[:, q + k:].clone().requires_grad_())
    O64 = [core_of_shard(QK64, V64, i, m) for i in range(2)]
    X264 = X64 + sum(o.detach() @ c(w) for o, w in zip(O64, WO))
    w1, w2 = torch.cat([c(w) for w in W1], 1), torch.cat([c(w) for w in W2], 0)
    A = X264 @ w1
    if act == "swiglu":
        w3 = torch.cat([c(w) for w in W3], 1)
        H = (X264 @ w3) * A * torch.sigmoid(A)
    else:
        H = A * 0.5 * torch.erfc(-A / 2 ** 0.5)
    Y64 = H @ w2
    vals = lambda buf, w: torch.from_numpy(ref.values(*ref.split(buf.cpu().numpy(), T, w), w))
    a8 = [vals(b, w) for b, w in zip(ckpt, WIDTHS * 2)]
    A8, dH = torch.cat(a8[:2], 1), c(dY) @ w2.T
    if act == "swiglu":
        U8, s = torch.cat(a8[2:], 1), torch.sigmoid(A8)
        H8, dU, dA = U8 * A8 * s, dH * A8 * s, dH * U8 * s * (1 + A8 * (1 - s))
        dX2 = dA @ w1.T + dU @ w3.T
    else:
        cdf = 0.5 * torch.erfc(-A8 / 2 ** 0.5)
        H8, dA = A8 * cdf, dH * (cdf + A8 * torch.exp(-A8 * A8 / 2) / (2 * np.pi) ** 0.5)
        dX2 = dA @ w1.T
    torch.autograd.backward(O64, [dX2 @ c(w).T for w in WO])
    dQKV64, dg64 = [], [0, 0]
    for i, (q, k) in enumerate(zip(DQ, DKV)):
        x = vals(kept[i], q + 2 * k)
        parts = []
        for j, (o, w, gain) in enumerate(((0, q, gq), (q, k, gk))):
            dx, dg = ref.heads_backward(heads(x[:, o:o + w]), heads(QK64[i].grad[:, o:o + w]), p, freq, "halves",
                                        c(gain).numpy(), 1e-6)[:2]
            parts.append(torch.from_numpy(dx.reshape(T, -1)))
            dg64[j] = dg64[j] + dg
        dQKV64.append(torch.cat(parts + [V64[i].grad], 1))
    want = {"Y": Y64, "dX": dX2 + sum(x @ c(w).T for x, w in zip(dQKV64, Wqkv)),
            "dW1": X264.T @ dA, "dW2": H8.T @ c(dY), "dWO": torch.cat([o.detach().T @ dX2 for o in O64]),
            "dWqkv": torch.cat([X64.T @ x for x in dQKV64], 1), "dgq": torch.from_numpy(dg64[0]),
            "dgk": torch.from_numpy(dg64[1])}
    got = {"Y": c(Y), "dX": c(dX), "dW1": torch.cat([c(x) for x in g["dW1"]], 1),
           "dW2": torch.cat([c(x) for x in g["dW2"]]), "dWO": torch.cat([c(x) for x in dWO]),
           "dWqkv": torch.cat([c(x) for x in dWqkv], 1), "dgq": c(dgq), "dgk": c(dgk)}
    errs = {k: ((got[k] - want[k]).abs().max() / want[k].abs().max()).item() for k in want}
    bad = {k: v for k, v in errs.items() if not v <= TOL}
    assert not bad, f"over {TOL}: {bad} (all {errs})"
