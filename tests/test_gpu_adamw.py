"""GPU parity of the AdamW step, the 8-bit states and the gradients' norm with the
oracle.

m and v (one fp32 rounding per operation) and their 8-bit codes are compared bit for
bit.  A weight: m / denom with the root, the two products, the addition, the
reciprocal or division (at most 2 ulp each for root and reciprocal) and the rate's
own rounding is within 16 u of itself, the decay and the last subtraction add 3 u of
the weight, u = 2^-24.  bf16 weights rounded from an fp32 copy: one storage
rounding; rounded randomly: the bits that the dither gives for some value within the
bound.
"""

import numpy as np
import pytest

from oracle.adamw import decode as state_decode
from oracle.adamw import encode, grad_norm, moments, random_bits, round_randomly, weights
from oracle.numerics import decode, round_to_storage

from gpu_util import assert_bitwise, from_dev, to_dev, torch_dtype

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

U = 2.0 ** -24
HYPER = dict(beta1=0.9, beta2=0.95, eps=1e-8)
# below, at and past 8 elements of a lane, blocks of 32, chunks of 2048
SIZES = [1, 2, 7, 8, 9, 31, 32, 33, 63, 100, 256, 511, 1000, 2047, 2048, 2049, 4100]


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def _storage(a, dtype):
    return round_to_storage(np.asarray(a, np.float64), dtype) if dtype == "bf16" else np.asarray(a, np.float32)


class Case:
    """Random tensors of one kind, on the host and on the GPU."""

    def __init__(self, sizes, dtype, grad, bits, master, seed, first=False, offset=0, decay=0.1):
        import torch
        rng = np.random.default_rng(seed)
        self.dtype, self.grad, self.bits, self.sizes = dtype, grad, bits, sizes
        self.decay = [decay] * len(sizes) if isinstance(decay, float) else decay
        self.w, self.x, self.g, self.m, self.v, self.ms, self.vs = [], [], [], [], [], [], []
        for n in sizes:
            full = (0.05 * rng.standard_normal(n)).astype(np.float32)
            self.w.append(_storage(full, dtype))
            self.x.append(full if master else None)
            size = np.exp(2 * rng.standard_normal(-(-n // 16))).repeat(16)[:n] * 1e-3
            g = size * rng.standard_normal(n)
            g[rng.random(n) < 0.05] = 0.0
            self.g.append(_storage(g, grad))
            m = np.zeros(n, np.float32) if first else (0.3 * size * rng.standard_normal(n)).astype(np.float32)
            v = np.zeros(n, np.float32) if first else (size * size * rng.random(n)).astype(np.float32)
            if bits == 8:
                half = np.full(n, 0x8000, np.uint32)
                m, a = encode(m, half, 16)
                v, b = encode(v, half, 32)
                self.ms.append(a)
                self.vs.append(b)
            self.m.append(m)
            self.v.append(v)

        def place(a, dt=None):
            # `offset` elements into a larger buffer, so that nothing is 16-byte aligned
            t = _dev(a) if dt is None else to_dev(a, dt)
            wide = torch.zeros(t.numel() + offset, dtype=t.dtype, device="cuda:0")
            wide[offset:].copy_(t)
            return wide[offset:]

        eight = bits == 8
        self.opt = tw.TwellAdamW([place(a, dtype) for a in self.w], [place(a) for a in self.m], [place(a) for a in self.v],
                                 [place(a) for a in self.ms] if eight else None,
                                 [place(a) for a in self.vs] if eight else None,
                                 [place(a) for a in self.x] if master else None, self.decay)
        self.grads = [place(a, grad) for a in self.g]

    def values(self, i):
        if self.bits == 32:
            return self.m[i], self.v[i]
        return (state_decode(self.m[i], self.ms[i], 16).astype(np.float32),
                state_decode(self.v[i], self.vs[i], 32).astype(np.float32))

    def check(self, step, lr, factor=None, seed=0, hyper=HYPER):
        """The GPU's tensors against one oracle step of the host's, which then take the GPU's place."""
        for i, n in enumerate(self.sizes):
            m0, v0 = self.values(i)
            m, v = moments(m0, v0, decode(self.g[i], self.grad), hyper["beta1"], hyper["beta2"], factor)
            bits = random_bits(seed + step, i, n)
            gm, gv = self.opt.m[i].cpu().numpy(), self.opt.v[i].cpu().numpy()
            if self.bits == 32:
                assert_bitwise(gm, m, f"m[{i}]")
                assert_bitwise(gv, v, f"v[{i}]")
            else:
                code, byte = encode(m, bits & 0xFFFF, 16)
                assert_bitwise(self.opt.m_scale[i].cpu().numpy(), byte, f"m_scale[{i}]")
                assert_bitwise(gm, code, f"m[{i}]")
                self.ms[i] = byte
                code, byte = encode(v, bits >> 16, 32)
                assert_bitwise(self.opt.v_scale[i].cpu().numpy(), byte, f"v_scale[{i}]")
                assert_bitwise(gv, code, f"v[{i}]")
                self.vs[i] = byte
            self.m[i], self.v[i] = gm, gv
            w0 = decode(self.w[i], self.dtype) if self.x[i] is None else self.x[i]
            w = weights(w0, m, v, lr, step, hyper["beta1"], hyper["beta2"], hyper["eps"], self.decay[i])
            kept = (1 - lr * self.decay[i]) * np.asarray(w0, np.float64)
            bound = 16 * U * np.abs(w - kept) + 3 * U * (np.abs(kept) + np.abs(w)) + 2.0 ** -148
            got = from_dev(self.opt.weights[i], self.dtype)
            if self.x[i] is not None:
                x = self.opt.master[i].cpu().numpy()
                assert (np.abs(x - w) <= bound).all(), f"master[{i}]"
                assert_bitwise(got, round_to_storage(x.astype(np.float64), "bf16"), f"w[{i}]")
                self.x[i] = x
            elif self.dtype == "f32":
                assert (np.abs(got - w) <= bound).all(), f"w[{i}]"
            else:
                # the random rounding of the bound's ends, in the order of the values
                ends = [decode(round_randomly((w + s * bound).astype(np.float32), bits), "bf16") for s in (-1, 1)]
                value = decode(got, "bf16")
                assert ((np.minimum(*ends) <= value) & (value <= np.maximum(*ends))).all(), f"w[{i}]"
            self.w[i] = got


KINDS = [("f32", "f32", 32, False), ("f32", "f32", 8, False), ("f32", "bf16", 8, False), ("bf16", "f32", 32, True),
         ("bf16", "bf16", 32, False), ("bf16", "f32", 8, False), ("bf16", "bf16", 8, True), ("f32", "bf16", 32, False),
         ("bf16", "bf16", 32, True), ("bf16", "f32", 32, False), ("bf16", "f32", 8, True), ("bf16", "bf16", 8, False)]


@pytest.mark.parametrize("dtype,grad,bits,master", KINDS)
@pytest.mark.parametrize("offset", [0, 1])
def test_steps(dtype, grad, bits, master, offset):
    print(f"step {dtype} grad {grad} bits {bits} master {master} offset {offset}", flush=True)
    c = Case(SIZES, dtype, grad, bits, master, 1, offset=offset)
    for t in (7, 8):
        tw.twell_adamw_step(c.opt, c.grads, lr=1e-3, step=t, **HYPER)
        c.check(t, 1e-3)


@pytest.mark.parametrize("dtype,grad,bits,master", KINDS[:6])
def test_first_steps_from_zeros(dtype, grad, bits, master):
    c = Case([100, 33], dtype, grad, bits, master, 2, first=True)
    for t in (1, 2, 3):
        tw.twell_adamw_step(c.opt, c.grads, lr=1e-2, step=t, seed=(5 << 32) + 9, **HYPER)
        c.check(t, 1e-2, seed=(5 << 32) + 9)


def test_zeros_makes_the_states_before_the_first_step():
    import torch
    w = [torch.randn(5, 33, device="cuda:0").bfloat16(), torch.randn(100, device="cuda:0")]
    g = [torch.randn_like(t) for t in w]
    for bits in (32, 8):
        opt = tw.TwellAdamW.zeros([t.clone() for t in w], bits=bits, master=True, weight_decay=[0.1, 0.0])
        assert opt.master[0].dtype == torch.float32 and opt.master[1] is None
        tw.twell_adamw_step(opt, g, lr=0.125, step=1, eps=0.0)
        # the first step moves every weight by lr against its gradient's sign
        for i, keep in ((0, 1 - 0.125 * 0.1), (1, 1.0)):
            x = opt.master[0] if i == 0 else opt.weights[1]
            want = w[i].double() * keep - 0.125 * torch.sign(g[i].double())
            assert ((x - want).abs() <= 32 * U * (want.abs() + 0.125)).all()
        if bits == 8:
            m, v = tw.twell_adamw_states(opt)
            assert m[0].shape == w[0].shape and v[1].dtype == torch.bfloat16


def test_mixed_list_and_many_tensors():
    # more tensors than a launch holds, of every kind in one list, with a decay each;
    # the random bits go by the place in the whole list
    import torch
    sizes = [int(n) for n in np.random.default_rng(3).integers(1, 300, 110)]
    decay = [0.1 * (i % 3) for i in range(110)]
    one = Case(sizes, "f32", "f32", 8, False, 4, decay=decay)
    tw.twell_adamw_step(one.opt, one.grads, lr=1e-3, step=11, **HYPER)
    one.check(11, 1e-3)
    kinds = [Case([200 + i], *KINDS[i], 5 + i) for i in range(12)]
    cat = lambda name: [getattr(k.opt, name)[0] for k in kinds]  # noqa: E731
    opt = tw.TwellAdamW(cat("weights"), cat("m"), cat("v"), cat("m_scale"), cat("v_scale"), cat("master"), 0.1)
    alone = [tw.TwellAdamW([k.opt.weights[0].clone()], [k.opt.m[0].clone()], [k.opt.v[0].clone()],
                           None if k.bits == 32 else [k.opt.m_scale[0].clone()],
                           None if k.bits == 32 else [k.opt.v_scale[0].clone()],
                           [None if k.opt.master[0] is None else k.opt.master[0].clone()], 0.1) for k in kinds]
    tw.twell_adamw_step(opt, [k.grads[0] for k in kinds], lr=1e-3, step=9, **HYPER)
    for k, a in zip(kinds, alone):
        tw.twell_adamw_step(a, k.grads, lr=1e-3, step=9, **HYPER)
        if k.bits == 32:
            assert torch.equal(k.opt.m[0], a.m[0]) and torch.equal(k.opt.v[0], a.v[0])
            if k.dtype == "f32":
                assert torch.equal(k.opt.weights[0], a.weights[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_clip_and_norm(bits):
    c = Case([1000, 2049, 1, 33], "f32", "f32", bits, False, 6)
    for max_norm in (1e-3, 1e3):
        clip = tw.twell_grad_norm(c.grads, max_norm)
        norm, factor = grad_norm([decode(g, "f32") for g in c.g], max_norm)
        got = clip.cpu().numpy()
        # one rounding of the norm; the factor: that, the limit's own rounding and the division's
        assert abs(got[0] - norm) <= U * norm * (1 + 1e-6) and abs(got[1] - factor) <= 3 * U * factor * (1 + 1e-6)
        t = 5 if max_norm < 1 else 6
        tw.twell_adamw_step(c.opt, c.grads, lr=1e-3, step=t, clip=clip, **HYPER)
        c.check(t, 1e-3, factor=got[1])


@pytest.mark.parametrize("sizes,grad", [([1], "f32"), ([0, 5, 0], "bf16"), ([4096, 4097, 9000], "f32"),
                                        ([100] * 200, "bf16"), ([3000001], "bf16"), ([9000000, 11], "f32")])
def test_grad_norm(sizes, grad):
    import torch
    rng = np.random.default_rng(len(sizes))
    g = [_storage(rng.standard_normal(n) * np.exp(3 * rng.standard_normal()), grad) for n in sizes]
    d = [to_dev(a, grad) for a in g]
    out = tw.twell_grad_norm(d, 0.5)
    norm, factor = grad_norm([decode(a, grad) for a in g], 0.5)
    got = out.cpu().numpy()
    assert abs(got[0] - norm) <= U * norm * (1 + 1e-6) and abs(got[1] - factor) <= 3 * U * factor * (1 + 1e-6)
    assert torch.equal(out, tw.twell_grad_norm(d, 0.5))
    # views of one flat buffer, at odd places
    flat = torch.cat([torch.zeros(1, dtype=d[0].dtype, device="cuda:0")] + d)
    at, views = 1, []
    for t in d:
        views.append(flat[at:at + t.numel()])
        at += t.numel()
    assert torch.equal(tw.twell_grad_norm(views, 0.5)[0], out[0]) or abs(float(tw.twell_grad_norm(views, 0.5)[0]) - norm) <= U * norm * (1 + 1e-6)


def test_norms_at_the_ends_of_the_range():
    import torch
    t = lambda *v: [torch.tensor(v, device="cuda:0")]  # noqa: E731
    assert tw.twell_grad_norm(t(3e38, -1e38), 1.0)[0].item() == np.float32(np.hypot(float(np.float32(3e38)), float(np.float32(1e38))))
    assert tw.twell_grad_norm(t(1e-45, 0.0), 1.0).tolist() == [np.float32(1e-45), 1.0]
    assert tw.twell_grad_norm(t(0.0), 1.0).tolist() == [0.0, 1.0]
    assert tw.twell_grad_norm(t(2.0)).tolist() == [2.0, 1.0]
    for bad in ((float("inf"),), (1.0, float("nan")), (3.4e38, 3.4e38)):
        out = tw.twell_grad_norm(t(*bad), 1.0)
        assert not np.isfinite(out[0].item()) and np.isnan(out[1].item())


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite_leave_the_step_out(bits):
    import torch
    c = Case([70, 5], "f32", "f32", bits, False, 7)
    before = [t.clone() for t in c.opt.weights + c.opt.m + c.opt.v]
    c.grads[1][3] = float("inf")
    clip = tw.twell_grad_norm(c.grads, 1.0)
    tw.twell_adamw_step(c.opt, c.grads, lr=1e-3, step=3, clip=clip)
    assert all(torch.equal(a, b) for a, b in zip(before, c.opt.weights + c.opt.m + c.opt.v))
    # without a clip it reaches its own element, and in 8 bits its own block
    tw.twell_adamw_step(c.opt, c.grads, lr=1e-3, step=3)
    assert torch.isfinite(c.opt.weights[0]).all() and torch.isfinite(c.opt.weights[1][[0, 1, 2, 4]]).all()
    if bits == 8:
        m, v = tw.twell_adamw_states(c.opt, torch.float32)
        assert torch.isnan(m[1]).all() and torch.isnan(v[1]).all() and torch.isfinite(m[0]).all()


def test_states_of_every_size():
    # blocks from the smallest scale to the largest and past it, zeros, one element far
    # below its block
    n = 32 * 300
    rng = np.random.default_rng(8)
    g = rng.standard_normal((300, 32)) * np.exp2(np.linspace(-149, 66, 300))[:, None]
    g[5], g[6, 1:] = 0.0, 0.0
    g[10:40, 3] *= 2.0 ** -20
    g = g.astype(np.float32).reshape(-1)
    import torch
    opt = tw.TwellAdamW.zeros([torch.zeros(n, device="cuda:0")], bits=8)
    tw.twell_adamw_step(opt, [_dev(g)], lr=1e-3, step=1, **HYPER)
    m, v = moments(np.zeros(n), np.zeros(n), g, 0.9, 0.95)
    bits = random_bits(1, 0, n)
    for got, scale, x, r, fields in ((opt.m, opt.m_scale, m, bits & 0xFFFF, 16), (opt.v, opt.v_scale, v, bits >> 16, 32)):
        code, byte = encode(x, r, fields)
        assert_bitwise(scale[0].cpu().numpy(), byte, "scales")
        assert_bitwise(got[0].cpu().numpy(), code, "codes")
    assert (opt.v_scale[0] == 255).any() and (opt.v_scale[0] == 40).any()
    for dtype in ("f32", "bf16"):
        rm, rv = tw.twell_adamw_states(opt, torch_dtype(dtype))
        for got, code, byte, fields in ((rm, opt.m, opt.m_scale, 16), (rv, opt.v, opt.v_scale, 32)):
            want = state_decode(code[0].cpu().numpy(), byte[0].cpu().numpy(), fields)
            assert np.array_equal(decode(from_dev(got[0], dtype), dtype), want, equal_nan=True)


def test_reading_every_code_and_scale():
    import torch
    code = np.tile(np.arange(256, dtype=np.uint8), 256)
    byte = np.repeat(np.arange(256, dtype=np.uint8), 8)
    n = code.size
    opt = tw.TwellAdamW([torch.zeros(n - 3, device="cuda:0")], [_dev(code)[:n - 3]], [_dev(code)[:n - 3]], [_dev(byte)],
                        [_dev(byte)])
    m, v = tw.twell_adamw_states(opt, torch.float32)
    for got, fields in ((m, 16), (v, 32)):
        want = state_decode(code, byte, fields)[:n - 3]
        assert np.array_equal(got[0].cpu().numpy().astype(np.float64), want, equal_nan=True)


@pytest.mark.parametrize("what", ["m", "v", "w"])
def test_small_steps_count_in_the_mean(what):
    # 200 steps that are each far smaller than half the distance between two codes (or
    # two bf16 numbers).  A step's rounding is off by at most one distance d, a
    # variance of at most d^2 / 4; d is at most 1/8 of the value (1/128 for bf16), so
    # after 200 steps an element is within sqrt(200) / 16 (/ 256) of the value in the
    # mean square, and the mean of 2^16 within 6 / 2^8 of that.
    import torch
    n, steps = 1 << 16, 200
    ones = torch.ones(n, device="cuda:0")
    zero = torch.zeros(n, device="cuda:0")
    if what == "w":
        opt = tw.TwellAdamW.zeros([ones.bfloat16()])
        for t in range(1, steps + 1):
            tw.twell_adamw_step(opt, [ones], lr=2.0 ** -13, step=t, eps=0.0)
        want, got, relative = 1 - steps * 2.0 ** -13, opt.weights[0].double().mean().item(), 1 / 256
    else:
        opt = tw.TwellAdamW.zeros([ones.clone()], bits=8)
        code, byte = encode(np.ones(32, np.float32), np.zeros(32, np.uint32), 16 if what == "m" else 32)
        getattr(opt, what)[0].fill_(int(code[0]))
        getattr(opt, f"{what}_scale")[0].fill_(int(byte[0]))
        for t in range(1, steps + 1):
            tw.twell_adamw_step(opt, [zero], lr=0.0, step=t, beta1=0.998, beta2=0.998)
        want = 0.998 ** steps
        got = tw.twell_adamw_states(opt, torch.float32)[0 if what == "m" else 1][0].double().mean().item()
        relative = 1 / 16
    assert abs(got - want) <= want * np.sqrt(steps) * relative * 6 / 2 ** 8
    # and rounding to nearest would not have moved at all
    assert abs(got - 1.0) > abs(got - want)


@pytest.mark.parametrize("bits", [32, 8])
def test_capture_with_step_and_rate_on_the_gpu(bits):
    import torch
    c, d = (Case([3000, 33], "bf16", "f32", bits, False, 9) for _ in range(2))
    step = torch.tensor([4], dtype=torch.int64, device="cuda:0")
    lr = torch.tensor([1e-3], device="cuda:0")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    clip = tw.twell_grad_norm(c.grads, 1e-2)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda:0")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        step.add_(1)
        tw.twell_grad_norm(c.grads, 1e-2, out=clip, workspace=ws)
        tw.twell_adamw_step(c.opt, c.grads, lr=lr, step=step, clip=clip, **HYPER)
    for t in (5, 6, 7):
        rate = float(np.float32(1e-3 / t))
        lr.fill_(rate)
        for g, h in zip(c.grads, d.grads):
            g.mul_(0.5)
            h.mul_(0.5)
        graph.replay()
        tw.twell_adamw_step(d.opt, d.grads, lr=rate, step=t, clip=tw.twell_grad_norm(d.grads, 1e-2), **HYPER)
        torch.cuda.synchronize()
        for name in ("weights", "m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
            assert all(torch.equal(a, b) for a, b in zip(getattr(c.opt, name), getattr(d.opt, name))), (t, name)
    # a step below 1 is left out
    before = [w.clone() for w in c.opt.weights]
    tw.twell_adamw_step(c.opt, c.grads, lr=lr, step=torch.zeros(1, dtype=torch.int64, device="cuda:0"))
    assert all(torch.equal(a, b) for a, b in zip(before, c.opt.weights))


@pytest.mark.parametrize("bits,dtype", [(8, "bf16"), (32, "f32")])
def test_offsets_beyond_32_bits(bits, dtype):
    # more than 2^31 elements (2^32 bytes of bf16 and more): the last chunk is stepped as
    # a tensor of its own would be, but for its random bits
    import torch
    n = (1 << 31) + 2048 + 5
    w = torch.zeros(n, dtype=torch_dtype(dtype), device="cuda:0")
    opt = tw.TwellAdamW.zeros([w], bits=bits, weight_decay=0.5)
    tail = 4101
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda:0")
    g[-tail:] = torch.randn(tail, device="cuda:0")
    w[-tail:] = torch.randn(tail, device="cuda:0")
    small = tw.TwellAdamW.zeros([w[-tail - 32:].float()], weight_decay=0.5)
    tw.twell_adamw_step(opt, [g], lr=0.1, step=1)
    tw.twell_adamw_step(small, [g[-tail - 32:].contiguous()], lr=0.1, step=1)
    assert not opt.weights[0][:1 << 20].any()
    got, want = opt.weights[0][-tail - 32:].double(), small.weights[0].double()
    # one step between bf16 numbers
    assert ((got - want).abs() <= want.abs() * (2.0 ** -7 if dtype == "bf16" else 4 * U) + 2.0 ** -100).all()
    assert abs(float(tw.twell_grad_norm([g])[0]) - float(g[-tail:].double().norm())) <= 1e-6 * float(g[-tail:].double().norm())
    if bits == 8:
        m = tw.twell_adamw_states(opt)[0][0][-tail:].double()
        assert ((m - 0.1 * g[-tail:].double()).abs() <= 0.1 * g[-tail:].double().abs() / 8 + 2.0 ** -16).all()


def test_binding_refuses():
    import torch
    c = Case([40, 50], "bf16", "f32", 8, False, 10)
    o = c.opt
    cpu = [g.cpu() for g in c.grads]
    for call in (lambda: tw.twell_adamw_step(o, c.grads[:1], lr=1e-3, step=1),
                 lambda: tw.twell_adamw_step(o, [c.grads[0], c.grads[0]], lr=1e-3, step=1),
                 lambda: tw.twell_adamw_step(o, cpu, lr=1e-3, step=1),
                 lambda: tw.twell_adamw_step(o, [None, c.grads[1]], lr=1e-3, step=1),
                 lambda: tw.twell_adamw_step(o, c.grads, lr=1e-3, step=0),
                 lambda: tw.twell_adamw_step(o, c.grads, lr=torch.ones(2, device="cuda:0"), step=1),
                 lambda: tw.twell_adamw_step(o, c.grads, lr=1e-3, step=1, clip=torch.ones(3, device="cuda:0")),
                 lambda: tw.twell_grad_norm([c.grads[0], cpu[1]]),
                 lambda: tw.twell_grad_norm([torch.zeros(4, 4, device="cuda:0").t()[:, :3]]),
                 lambda: tw.TwellAdamW(o.weights, o.m, o.v, o.m_scale, None),
                 lambda: tw.TwellAdamW(o.weights, o.m, o.v[:1], o.m_scale, o.v_scale),
                 lambda: tw.TwellAdamW(o.weights, o.m, o.v, o.v_scale, [s[:1] for s in o.v_scale]),
                 lambda: tw.TwellAdamW([w.float() for w in o.weights], o.m, o.v, o.m_scale, o.v_scale, [w.float() for w in o.weights]),
                 lambda: tw.TwellAdamW(o.weights, o.m, o.v, o.m_scale, o.v_scale, weight_decay=[0.1])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: tw.twell_adamw_step(o, [g.half() for g in c.grads], lr=1e-3, step=1),
                 lambda: tw.twell_adamw_step(o, c.grads, lr=1e-3, step=torch.ones(1, device="cuda:0")),
                 lambda: tw.TwellAdamW(o.weights, o.m, o.v)):
        with pytest.raises(TypeError):
            call()
    for kw in (dict(lr=-1.0), dict(lr=1e-3, beta1=1.0), dict(lr=1e-3, eps=float("nan"))):
        with pytest.raises(tw.TwellError):
            tw.twell_adamw_step(o, c.grads, step=1, **kw)
    with pytest.raises(tw.TwellError):
        tw.twell_grad_norm(c.grads, 0.0)


def test_tensors_that_share_memory_are_refused():
    import torch
    w = torch.zeros(4, 100, device="cuda:0")
    v = [torch.zeros(100, device="cuda:0") for _ in range(4)]
    one = tw.TwellAdamW([w[0], w[1]], v[:2], v[2:])  # side by side
    tw.twell_adamw_step(one, [v[0] + 1, v[0] + 1], lr=1e-3, step=1)
    empty = torch.zeros(0, device="cuda:0")
    tw.TwellAdamW([empty, empty, w[0]], [empty, empty, v[0]], [empty, empty, v[1]])
    flat = w.view(-1)
    for call in (lambda: tw.TwellAdamW([w[0], w[0]], v[:2], v[2:]), lambda: tw.TwellAdamW([w[0], w[1]], v[:2], v[:2]),
                 lambda: tw.TwellAdamW([w[0]], [w[0]], v[:1]), lambda: tw.TwellAdamW.zeros([w[0], flat[99:199]]),
                 lambda: tw.TwellAdamW.zeros([w, w], bits=8)):
        with pytest.raises(ValueError, match="share memory"):
            call()


def test_norm_refuses_a_missing_gradient():
    import torch
    g = torch.ones(3, device="cuda:0")
    for grads in ([None], [None, g], [g, None]):
        with pytest.raises(ValueError, match="required"):
            tw.twell_grad_norm(grads)


def test_norm_up_to_the_largest_number():
    # 2^128 - 2^104 is finite: so is its norm, and it is clipped as any other
    import torch
    top = float(np.finfo(np.float32).max)
    g = torch.tensor([top], device="cuda:0")
    assert tw.twell_grad_norm([g], 1024.0).tolist() == [top, float(np.float32(1024.0) / np.float32(top))]
    assert tw.twell_grad_norm([g]).tolist() == [top, 1.0]


def test_weights_from_a_generator_and_of_no_dimension():
    import torch
    layer = torch.nn.Linear(40, 3, device="cuda:0")
    scale = torch.nn.Parameter(torch.tensor(2.0, device="cuda:0"))
    for bits in (32, 8):
        weights = [*layer.parameters(), scale]
        opt = tw.TwellAdamW.zeros((w for w in weights), bits=bits)
        before = [w.detach().clone() for w in weights]
        tw.twell_adamw_step(opt, (torch.ones_like(w) for w in weights), lr=0.125, step=1, eps=0.0)
        # m / (1 - beta1) / sqrt(v / (1 - beta2)) = 1 but for the roundings of nine operations, 3 of them to 1 ulp
        for w, b in zip(weights, before):
            assert w.shape == b.shape and ((w - b + 0.125).abs() <= 0.125 * 16 * U + 2 * U * b.abs()).all()
        if bits == 8:
            m, v = tw.twell_adamw_states(opt)
            assert [t.shape for t in m] == [w.shape for w in weights]
