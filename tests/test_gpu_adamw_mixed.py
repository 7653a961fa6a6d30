"""One list of tensors of every kind: each is stepped with its own buffers, its own
decay and the random bits of its place in the whole list (8-bit states and
randomly rounded weights bit for bit, as in test_gpu_adamw.py)."""

import numpy as np
import pytest

import test_gpu_adamw
from oracle.adamw import encode, grad_norm, moments, random_bits
from oracle.numerics import decode
from test_gpu_adamw import HYPER, KINDS, U, Case

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

BUFFERS = ("weights", "m", "v", "m_scale", "v_scale", "master")


def _mixed(count, seed):
    """(a Case of one tensor for each place, the optimiser of all of them, their gradients)."""
    rng = np.random.default_rng(seed)
    kinds = [int(k) for k in rng.integers(0, len(KINDS), count)]
    for k in range(len(KINDS)):  # every kind, and more of the fifth than a launch takes
        kinds[k] = k
    kinds[len(KINDS):len(KINDS) + 45] = [5] * 45
    rng.shuffle(kinds)
    cases = [Case([int(rng.integers(1, 500))], *KINDS[k], 100 + i, offset=int(rng.integers(0, 2)), decay=0.1 * (i % 3))
             for i, k in enumerate(kinds)]
    opt = tw.TwellAdamW(*([getattr(c.opt, name)[0] for c in cases] for name in BUFFERS), [c.decay[0] for c in cases])
    return kinds, cases, opt, [c.grads[0] for c in cases]


@pytest.mark.parametrize("clipped", [False, True])
def test_each_tensor_by_its_place(clipped, monkeypatch):
    kinds, cases, opt, grads = _mixed(120, 1)
    before = [(c.values(0), c.g[0]) for c in cases]
    factor = clip = None
    if clipped:
        clip = tw.twell_grad_norm(grads, 0.01)
        norm, factor = grad_norm([decode(c.g[0], c.grad) for c in cases], 0.01)
        got = clip.cpu().numpy()
        assert abs(got[0] - norm) <= U * norm * (1 + 1e-6) and abs(got[1] - factor) <= 3 * U * factor * (1 + 1e-6)
        factor = got[1]
    tw.twell_adamw_step(opt, grads, lr=1e-3, step=9, seed=77, clip=clip, **HYPER)
    for place, c in enumerate(cases):
        monkeypatch.setattr(test_gpu_adamw, "random_bits", lambda seed, _, n: random_bits(seed, place, n))
        c.check(9, 1e-3, factor=factor, seed=77)
    # the bits of another place would show: those of the tensor's number among its kind
    differ = 0
    for place, (c, ((m0, v0), g)) in enumerate(zip(cases, before)):
        among = kinds[:place].count(kinds[place])
        if c.bits != 8 or among == place:
            continue
        m, v = moments(m0, v0, decode(g, c.grad), HYPER["beta1"], HYPER["beta2"], factor)
        bits = random_bits(77 + 9, among, c.sizes[0])
        differ += (not np.array_equal(encode(m, bits & 0xFFFF, 16)[0], c.m[0])
                   or not np.array_equal(encode(v, bits >> 16, 32)[0], c.v[0]))
    assert differ > 50


def test_states_of_a_mixed_list():
    # 8-bit states of every kind of weight, read back in one call
    from oracle.adamw import decode as state_decode
    kinds, cases, opt, grads = _mixed(120, 2)
    eight = [i for i, c in enumerate(cases) if c.bits == 8]
    part = tw.TwellAdamW(*([getattr(opt, name)[i] for i in eight] for name in BUFFERS))
    import torch
    m, v = tw.twell_adamw_states(part, torch.float32)
    for at, i in enumerate(eight):
        c = cases[i]
        for got, code, byte, fields in ((m[at], c.m[0], c.ms[0], 16), (v[at], c.v[0], c.vs[0], 32)):
            assert np.array_equal(got.cpu().numpy().astype(np.float64), state_decode(code, byte, fields))
    with pytest.raises(ValueError):
        tw.twell_adamw_states(opt)
