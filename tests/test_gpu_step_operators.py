"""The operators around the GEMM launches together, as a layer's training step uses them: norm, QKV projection, an
attention core (plain torch here), output projection with the residual stream in its epilogue, norm, MLP block with the
residual stream, all of it backward, and an AdamW step of every tensor with the gradients' norm clipped.

The reference runs the same formulas in 64 bits with torch's own gradients.  Tolerance: at most sixteen tensors rounded
to bf16 lie between an input and any result, each off by 2^-8 of its value: 16 * 2^-8 of the largest reference value."""
import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu

T, d, D = 160, 128, 64
DQ, DKV = [128, 64], [64, 64]
WIDTHS = [192, 72]
EPS = 1e-5
TOL = 16 * 2.0 ** -8


def core(q, k, v, mask):
    """Causal attention of [T, H, D] heads (grouped keys), elementary operations."""
    g = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("thd,shd->hts", q, k) / D ** 0.5
    p = torch.softmax(s.masked_fill(~mask, float("-inf")), -1)
    return torch.einsum("hts,shd->thd", p, v)


def core_of_shard(QKV, i, mask):
    split = lambda t: t.reshape(T, -1, D)
    q, k, v = QKV.split([DQ[i], DKV[i], DKV[i]], 1)
    return core(split(q), split(k), split(v), mask).reshape(T, -1)


def weights(act, seed=3):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=0.1: (torch.randn(*s, generator=gen) * std).bfloat16().cuda()
    w = {"g1": 1 + rnd(d), "c1": rnd(d), "g2": 1 + rnd(d), "c2": rnd(d)}
    w |= {f"Wqkv{i}": rnd(d, q + 2 * k) for i, (q, k) in enumerate(zip(DQ, DKV))}
    w |= {f"WO{i}": rnd(q, d) for i, q in enumerate(DQ)}
    w |= {f"W1{i}": rnd(d, n) for i, n in enumerate(WIDTHS)} | {f"W2{i}": rnd(n, d) for i, n in enumerate(WIDTHS)}
    if act == "swiglu":
        w |= {f"W3{i}": rnd(d, n) for i, n in enumerate(WIDTHS)}
    return w, rnd(T, d, std=1.0), rnd(T, d, std=1.0)


class Layer:
    def __init__(self, tp, act, kind):
        self.act, self.kind = act, kind
        self.norm1, self.norm2 = (tp.TokenNorm(T, d, kind, "bf16", eps=EPS) for _ in "12")
        self.proj = tp.ShardedAttentionProj(T, d, DQ, DKV, "bf16")
        self.mlp = tp.ShardedMLP(T, d, WIDTHS, act, "bf16")
        self.mask = torch.ones(T, T, device="cuda").tril().bool()

    def list_of(self, w, name):
        return [w[f"{name}{i}"] for i in range(2)] if f"{name}0" in w else None

    def step(self, w, X, dY):
        """Y and every gradient, by name."""
        L = self.list_of
        c1, c2 = (w["c1"], w["c2"]) if self.kind == "layer" else (None, None)
        bias = self.kind == "layer"
        N1, st1, _ = self.norm1.forward(X, w["g1"], c1)
        QKV = [x.float().requires_grad_() for x in self.proj.qkv_forward(N1, L(w, "Wqkv"))]
        O = [core_of_shard(x, i, self.mask) for i, x in enumerate(QKV)]
        Ob = [x.detach().bfloat16() for x in O]
        S = self.proj.out_forward(L(w, "WO"), Ob, residual=X)
        N2, st2, _ = self.norm2.forward(S, w["g2"], c2)
        Y, saved, H = self.mlp.forward(N2, L(w, "W1"), L(w, "W2"), L(w, "W3"), residual=S)

        g = self.mlp.backward(N2, L(w, "W1"), L(w, "W2"), saved, H, dY, L(w, "W3"))
        dS, dg2, dc2 = self.norm2.backward(S, st2, g["dX"], w["g2"], dsum=dY, bias_grad=bias)
        dO, dWO = self.proj.out_backward(L(w, "WO"), Ob, dS)
        dQKV = [x.bfloat16() for x in torch.autograd.grad(O, QKV, [x.float() for x in dO])]
        dN1, dWqkv = self.proj.qkv_backward(N1, L(w, "Wqkv"), dQKV)
        dX, dg1, dc1 = self.norm1.backward(X, st1, dN1, w["g1"], dsum=dS, bias_grad=bias)
        out = {"g1": dg1, "g2": dg2} | ({"c1": dc1, "c2": dc2} if bias else {})
        for name, xs in (("Wqkv", dWqkv), ("WO", dWO), ("W1", g["dW1"]), ("W2", g["dW2"]), ("W3", g["dW3"])):
            out |= {f"{name}{i}": x for i, x in enumerate(xs or [])}
        return Y, dX, out

    def reference(self, w, X, dY):
        w = {k: v.double().requires_grad_() for k, v in w.items()}
        X = X.double().requires_grad_()
        c1, c2 = (w["c1"], w["c2"]) if self.kind == "layer" else (None, None)
        N1 = ref.norm_forward(X, w["g1"], c1, self.kind, EPS)[0]
        S = X
        for i in range(2):
            S = S + core_of_shard(N1 @ w[f"Wqkv{i}"], i, self.mask) @ w[f"WO{i}"]
        N2 = ref.norm_forward(S, w["g2"], c2, self.kind, EPS)[0]
        Y = S
        for i in range(2):
            a = N2 @ w[f"W1{i}"]
            h = torch.nn.functional.silu(a) * (N2 @ w[f"W3{i}"]) if self.act == "swiglu" else \
                torch.nn.functional.gelu(a)
            Y = Y + h @ w[f"W2{i}"]
        names = [k for k in w if self.kind == "layer" or k not in ("c1", "c2")]
        grads = torch.autograd.grad(Y, [X] + [w[k] for k in names], dY.double())
        return Y.detach(), grads[0], dict(zip(names, grads[1:]))


@pytest.mark.parametrize("act,kind", [("gelu", "layer"), ("swiglu", "rms")])
def test_gradients_of_a_layer(gpu_lib, act, kind):
    w, X, dY = weights(act)
    layer = Layer(gpu_lib, act, kind)
    Y, dX, g = layer.step(w, X, dY)
    Y64, dX64, g64 = layer.reference(w, X, dY)
    assert set(g) == set(g64)
    for name, a, b in [("Y", Y, Y64), ("dX", dX, dX64)] + [(k, g[k], g64[k]) for k in g]:
        err = (a.double() - b).abs().max() / b.abs().max()
        assert err <= TOL, (name, err.item())
    layer.mlp.check()
    layer.proj.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps_eager_and_captured(gpu_lib, bits):
    """Three steps of the layer with AdamW and clipping, then the same as one captured graph replayed: bit for bit the
    same weights and moments, and the weights moved against the gradient."""
    def run(captured):
        w, X, dY = weights("swiglu")
        layer = Layer(gpu_lib, "swiglu", "rms")
        names = [k for k in w if k not in ("c1", "c2")]
        opt = gpu_lib.ShardedAdamW([w[k] for k in names], lr=1e-2, weight_decay=0.01, bits=bits, master=True,
                                   max_norm=1.0, seed=5, capturable=True)

        def step():
            Y, _, g = layer.step(w, X, dY)
            return Y, g, opt.step([g[k] for k in names])

        start = [x.clone() for x in opt.master]
        Y, g, norm = step()
        first = {k: x.clone() for k, x in g.items()}
        if captured:
            torch.cuda.synchronize()
            del Y, g
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
            graph.replay()
        else:
            step()
            step()
        torch.cuda.synchronize()
        assert opt.steps == 3 and norm.item() > 1.0
        for k, a, b in zip(names, start, opt.master):
            assert ((b - a).double() * first[k].double()).sum() < 0, k
        m, v = opt.moments()
        layer.mlp.check()
        layer.proj.check()
        return opt.params + opt.master + m + v

    for a, b in zip(run(False), run(True)):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_two_captured_graphs_of_one_norm(gpu_lib):
    """Two graphs that share a norm's workspace, replayed in turn on one stream."""
    x = torch.randn(500, 512, device="cuda").bfloat16()
    g = torch.ones(512, device="cuda").bfloat16()
    norm = gpu_lib.TokenNorm(500, 512, "layer", "bf16")
    dys = [torch.randn(500, 512, device="cuda").bfloat16() for _ in "ab"]
    y, stats, _ = norm.forward(x, g)
    want = [norm.backward(x, stats, dy, g, bias_grad=True) for dy in dys]
    torch.cuda.synchronize()
    graphs, got = [], []
    for dy in dys:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(norm.backward(x, stats, dy, g, bias_grad=True))
        graphs.append(graph)
    for k in (0, 1, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
