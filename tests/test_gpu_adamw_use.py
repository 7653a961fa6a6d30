"""The optimiser as a training loop uses it: parameters of a module with autograd's
gradients, a graph from before a step, states that are put in place on resuming."""

import pytest

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")


def _model(dtype):
    import torch
    torch.manual_seed(3)
    return torch.nn.Sequential(torch.nn.Linear(40, 33), torch.nn.Linear(33, 5)).to("cuda:0", dtype)


def _grads(model, seed):
    import torch
    x = torch.randn(7, 40, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(seed))
    model.zero_grad()
    model(x.to(model[0].weight.dtype)).square().mean().backward()
    return [p.grad for p in model.parameters()]


@pytest.mark.parametrize("bits,master", [(32, False), (32, True), (8, False), (8, True)])
def test_a_resumed_run_goes_on_as_the_first(bits, master):
    import torch
    one, two = _model(torch.bfloat16), _model(torch.bfloat16)
    opts = [tw.TwellAdamW.zeros(m.parameters(), bits=bits, master=master, weight_decay=0.1) for m in (one, two)]
    for t in (1, 2, 3, 4):
        for m, o in zip((one, two), opts):
            g = _grads(m, t)
            tw.twell_adamw_step(o, g, lr=1e-2, step=t, clip=tw.twell_grad_norm(g, 0.5))
        # the second run ends here and goes on with copies of everything in other memory
        for p in two.parameters():
            p.data = p.data.clone()
        for name in ("m", "v", "m_scale", "v_scale", "master"):
            setattr(opts[1], name, [None if a is None else a.clone() for a in getattr(opts[1], name)])
        assert all(torch.equal(a, b) for a, b in zip(one.parameters(), two.parameters())), t
    for name in ("m", "v", "m_scale", "v_scale", "master"):
        for a, b in zip(getattr(opts[0], name), getattr(opts[1], name)):
            assert (a is None) == (b is None) and (a is None or torch.equal(a, b)), name
    if bits == 8:
        for a, b in zip(*(sum(tw.twell_adamw_states(o), []) for o in opts)):
            assert torch.equal(a, b)


def test_a_graph_from_before_the_step_is_refused():
    import torch
    model = _model(torch.float32)
    opt = tw.TwellAdamW.zeros(model.parameters())
    x = torch.ones(2, 40, device="cuda:0")
    g = _grads(model, 0)
    old = model(x).sum()
    tw.twell_adamw_step(opt, g, lr=1e-3, step=1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        old.backward()
    model(x).sum().backward()


def test_gradients_in_written_memory_are_refused():
    import torch
    flat = torch.zeros(300, device="cuda:0")
    opt = tw.TwellAdamW.zeros([flat[:100], flat[100:200]])
    tw.twell_adamw_step(opt, [flat[200:], flat[200:]], lr=1e-3, step=1)
    for bad in (flat[:100], flat[99:199], flat[199:299], opt.m[1], opt.v[0]):
        with pytest.raises(ValueError, match="share memory"):
            tw.twell_adamw_step(opt, [bad, flat[200:]], lr=1e-3, step=2)
    assert not flat.any()


def test_states_of_another_size_or_place_are_refused():
    import torch
    w = [torch.ones(64, device="cuda:0")]
    for bits in (32, 8):
        opt = tw.TwellAdamW.zeros(w, bits=bits)
        good = opt.m
        for bad in ([good[0].cpu()], [good[0][:63]], [good[0].half()], []):
            opt.m = bad
            with pytest.raises((ValueError, TypeError)):
                tw.twell_adamw_step(opt, [torch.ones(64, device="cuda:0")], lr=1e-3, step=1)
        opt.m = good
        tw.twell_adamw_step(opt, [torch.zeros(64, device="cuda:0")], lr=1e-3, step=1)
    assert torch.equal(w[0], torch.ones_like(w[0]))
