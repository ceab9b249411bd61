"""Rotation of part of a head, without a norm: an element from rotary_dim on is passed through by both passes, so a
NaN or an infinity there stays where it is."""
import pytest
import torch

from test_gpu_qk_norm_rope import make, proj_of

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32, "pairs"), (64, 32, "halves"), (96, 24, "halves"), (80, 20, "halves"), (64, 0, "halves"),
          (64, 0, "pairs"), (256, 64, "pairs"), (20, 10, "halves"), (20, 10, "pairs"), (250, 126, "halves"),
          (254, 100, "pairs"), (64, 6, "pairs"), (128, 96, "halves"), (2, 0, "pairs")]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,R,layout", SHAPES)
def test_special_values_stay_in_their_element(gpu_lib, D, R, layout, dtype):
    m = 8 if D % 8 else 1
    T = 70
    s = make(T, [2 * m], [m], D, dtype, seed=D + R)
    p = proj_of(gpu_lib, T, s, dtype, D, rotary_dim=R, layout=layout, norm=False)
    forward = lambda x: p.qk_norm_rope_forward([x], s["pos"])[0]
    backward = lambda y: p.qk_norm_rope_backward([torch.zeros_like(s["QKV"][0])], [y], s["pos"], dV_i=s["dV"])[0][0]
    n = 3 * m * D  # query and key columns
    for call, x in ((forward, s["QKV"][0]), (backward, s["dQK"][0])):
        clean = call(x)[:, :n].clone()
        gen = torch.Generator().manual_seed(D)
        at = torch.zeros(T, n, dtype=torch.bool)
        for t in range(T):  # one element a token, past rotary_dim in some head
            h = torch.randint(0, 3 * m, (1,), generator=gen).item()
            at[t, h * D + torch.randint(R, D, (1,), generator=gen).item()] = True
        at = at.cuda()
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda")[torch.arange(T, device="cuda") % 3]
        spoiled = x.clone()
        spoiled[:, :n] = torch.where(at, bad[:, None].to(x.dtype), spoiled[:, :n])
        got = call(spoiled)[:, :n]
        assert torch.equal(got[~at], clean[~at])
        assert torch.equal(got[at].nan_to_num(5.0), spoiled[:, :n][at].nan_to_num(5.0))
        # and what is not rotated is the input itself
        rest = (torch.arange(n, device="cuda") % D) >= R
        assert torch.equal(clean[:, rest], x[:, :n][:, rest])
