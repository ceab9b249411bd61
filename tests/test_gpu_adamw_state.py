"""The optimizer's tensors, replaced between two steps: what the lists hold is what a step works on."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SIZES = [5, 300, 4096, 70_001]
HYPER = dict(lr=1e-3, eps=1e-8, weight_decay=0.1, max_norm=1.0)


def make(tp, bits, master, **kw):
    gen = torch.Generator(device="cuda").manual_seed(1)
    p = [torch.randn(n, generator=gen, device="cuda").bfloat16() for n in SIZES]
    g = [torch.randn(n, generator=gen, device="cuda").bfloat16() for n in SIZES]
    return tp.ShardedAdamW(p, bits=bits, master=master, **HYPER, **kw), g


def state(opt):
    return [*opt.params, *(opt.master or ()), *opt.m, *opt.v]


def by_item(xs, k, new):
    xs[k] = new


def by_data(xs, k, new):
    xs[k].data = new


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("replace", [by_item, by_data])
def test_replaced_tensors(gpu_lib, bits, capturable, replace):
    want, g = make(gpu_lib, bits, True, capturable=capturable)
    opt, _ = make(gpu_lib, bits, True, capturable=capturable)
    for _ in range(2):
        want.step(g)
    opt.step(g)
    old = {}
    for name in ("params", "master", "m", "v"):
        xs = getattr(opt, name)
        for k in (0, 3):
            old[name, k] = xs[k].detach()  # holds the memory
            replace(xs, k, xs[k].clone())
    kept = {at: x.clone() for at, x in old.items()}
    opt.step(g)
    assert all(torch.equal(a, b) for a, b in zip(state(want), state(opt)))
    assert all(torch.equal(x, kept[at]) for at, x in old.items())
    assert all(torch.equal(a, b) for xs, ys in zip(want.moments(), opt.moments()) for a, b in zip(xs, ys))


@pytest.mark.parametrize("bits", [32, 8])
def test_restored_lists(gpu_lib, bits):
    """A checkpoint taken after one step and put back after three."""
    opt, g = make(gpu_lib, bits, True)
    opt.step(g)
    kept = {name: [x.clone() for x in getattr(opt, name)] for name in ("params", "master", "m", "v")}
    opt.step(g)
    want = [x.clone() for x in state(opt)]
    opt.step(g)
    opt.params, opt.master = tuple(kept["params"]), tuple(kept["master"])
    opt.load_moments(kept["m"], kept["v"], steps=1)
    opt.step(g)
    assert opt.steps == 2 and all(torch.equal(a, b) for a, b in zip(want, state(opt)))


@pytest.mark.parametrize("name", ["params", "master", "m", "v"])
def test_what_does_not_fit_is_refused(gpu_lib, name):
    opt, g = make(gpu_lib, 32, True)
    opt.step(g)
    before = [x.clone() for x in state(opt)]
    good = getattr(opt, name)[1]
    bad = [good.cpu(), good[:-1].clone(), good.double(), torch.stack([good, good], 1)[:, 0]]
    for x in bad:
        getattr(opt, name)[1] = x
        with pytest.raises(ValueError, match=name):
            opt.step(g)
    getattr(opt, name)[1] = good
    xs = getattr(opt, name)
    setattr(opt, name, xs[:-1])
    with pytest.raises(ValueError, match=name):
        opt.step(g)
    setattr(opt, name, xs)
    assert opt.steps == 1 and all(torch.equal(a, b) for a, b in zip(before, state(opt)))


def test_moments_of_replaced_tensors_are_read_out(gpu_lib):
    opt, g = make(gpu_lib, 8, False)
    opt.step(g)
    want = opt.moments()
    for xs in (opt.m, opt.v):
        new = xs[2].clone()
        xs[2].zero_()
        xs[2] = new
    assert all(torch.equal(a, b) for xs, ys in zip(want, opt.moments()) for a, b in zip(xs, ys))


def test_numbers_on_the_device_that_do_not_fit_are_refused(gpu_lib):
    opt, g = make(gpu_lib, 32, False, capturable=True)
    opt.step(g)
    before = [x.clone() for x in state(opt)]
    for name, good in (("lr_device", opt.lr_device), ("step_device", opt.step_device)):
        for bad in (good.cpu(), good.double(), good.int(), good.expand(2), good[None]):
            setattr(opt, name, bad)
            with pytest.raises(ValueError, match=name):
                opt.step(g)
        setattr(opt, name, good)
    assert opt.steps == 1 and all(torch.equal(a, b) for a, b in zip(before, state(opt)))
    opt.lr_device = torch.full((), 2e-3, device="cuda")  # another one that fits is taken
    opt.step(g)
    want, _ = make(gpu_lib, 32, False, capturable=True)
    want.step(g)
    want.lr_device.fill_(2e-3)
    want.step(g)
    assert all(torch.equal(a, b) for a, b in zip(state(want), state(opt)))
