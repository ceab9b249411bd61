"""The gains' gradients with the heads described anew: a graph captured before, and a call on another stream while the
current one is busy, both use the workspace that the object has had from the start."""
import pytest
import torch

from test_gpu_qk_norm_rope import make, proj_of

pytestmark = pytest.mark.gpu


def test_graph_captured_before(gpu_lib):
    s = make(300, [4], [4], 64, "fp32")
    p = proj_of(gpu_lib, 300, s, "fp32", 64)
    call = lambda g: p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], g, g, dV_i=s["dV"])
    want = call(s["gq"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(s["gq"])
    p.set_qk_norm_rope(256)
    others = [torch.full((1 << 22,), 7.0, device="cuda") for _ in range(4)]
    call(torch.ones(256, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want[0] + [want[1], want[2]], got[0] + [got[1], got[2]]):
        assert torch.equal(a, b)
    assert all((x == 7.0).all() for x in others)
    p.check()


def test_described_while_the_current_stream_is_busy(gpu_lib):
    s = make(300, [4], [4], 64, "fp32")
    p = proj_of(gpu_lib, 300, s, "fp32", 64)
    want = p.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], s["gq"], s["gk"], s["dV"])
    torch.cuda.synchronize()
    q = gpu_lib.ShardedAttentionProj(300, 64, s["dq"], s["dkv"], "fp32")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)  # about 10 ms
    q.set_qk_norm_rope(64, eps=1e-6)
    got = q.qk_norm_rope_backward(s["QKV"], s["dQK"], s["pos"], s["gq"], s["gk"], s["dV"], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(want[1], got[1]) and torch.equal(want[2], got[2])
