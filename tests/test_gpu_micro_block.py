"""The microscaled operators and the optimiser as a program uses them together:
serving with the gate in 4 bits and training steps of examples/ffn_block.py, against
the float64 oracle; captured graphs; two streams at once."""

import importlib.util
import os

import numpy as np
import pytest

from oracle.adamw import grad_norm, moments, weights
from oracle.block import norm_factor, residual_sum, rmsnorm
from oracle.ffn import ffn_from_h, rel_l2
from oracle.mx4 import matmul, quantize, unpack, values
from oracle.numerics import decode, round_to_storage
from oracle.twell import relu_storage
from workloads.synth import to_storage

from gpu_util import TOL, assert_bitwise, from_dev, to_dev, torch_dtype

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EPS = 1e-6
U = 2.0 ** -24


def _block(T, d, F, dtype, seed, cap=32, tile=128, density=0.02):
    import torch
    from statistics import NormalDist
    spec = importlib.util.spec_from_file_location("ffn_block", os.path.join(ROOT, "examples", "ffn_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    rng = np.random.default_rng(seed)
    s = {k: to_storage(v, dtype) for k, v in {
        "x": rng.standard_normal((T, d)), "res": rng.standard_normal((T, d)),
        "norm": 1.0 + 0.1 * rng.standard_normal(d), "wg": rng.standard_normal((F, d)) / d ** 0.5,
        "wu": rng.standard_normal((F, d)) / d ** 0.5, "wd": rng.standard_normal((F, d)) / F ** 0.5,
        "dy": rng.standard_normal((T, d)), "dh": rng.standard_normal((T, d))}.items()}
    dev = {k: to_dev(v, dtype) for k, v in s.items()}
    s["bias"] = np.full(T, NormalDist().inv_cdf(density), np.float32)
    dev["bias"] = torch.from_numpy(s["bias"]).to("cuda:0")
    return s, dev, ex.FfnBlock(dev["norm"], dev["wg"], dev["wu"], dev["wd"], EPS, tile=tile, cap=cap)


@pytest.mark.parametrize("dtype,T,d,F", [("f32", 67, 256, 512), ("bf16", 96, 512, 1024), ("bf16", 1, 512, 1024),
                                         ("bf16", 300, 512, 1024)])
def test_serving_block(dtype, T, d, F):
    s, dev, block = _block(T, d, F, dtype, 1)
    y, h = block.serve_mx4(dev["x"], dev["res"], dev["bias"])
    h_o = residual_sum(s["x"], s["res"], dtype)
    assert_bitwise(from_dev(h, dtype), h_o, "h")
    # the block from its definition: norm, its 4 bits, the product with the weights' 4
    # bits, then the layer with those gate activations
    z = (decode(h_o, dtype).astype(np.float32) * decode(s["norm"], dtype).astype(np.float32)).astype(np.float32)
    v = values(*quantize(z), factor=norm_factor(h_o, EPS, dtype))
    pre = round_to_storage(matmul(v, values(*quantize(decode(s["wg"], dtype))), s["bias"]), dtype)
    act = relu_storage(pre, dtype)
    n = round_to_storage(rmsnorm(h_o, s["norm"], EPS, dtype), dtype)
    want = ffn_from_h(decode(act, dtype), n, s["wu"], s["wd"], dtype)
    assert np.count_nonzero(decode(act, dtype) > 0, axis=1).max() > 0
    assert rel_l2(decode(from_dev(y, dtype), dtype), want) <= TOL[dtype]


@pytest.mark.parametrize("bits,master", [(32, True), (8, False), (32, False), (8, True)])
def test_training_steps(bits, master):
    dtype = "bf16"
    s, dev, block = _block(64, 512, 512, dtype, 2)
    opt = block.optimizer(bits, master)
    host = {n: [decode(from_dev(getattr(block, n), dtype), dtype).reshape(-1), 0.0, 0.0] for n in block.NAMES}
    for step in (1, 2, 3):
        grads = block.train_step(dev["x"], dev["res"], dev["dy"], dev["dh"], dev["bias"], width=64)[2]
        g = {n: grads[n].float().cpu().numpy().reshape(-1) for n in block.NAMES}
        clip = block.update(opt, grads, 1e-2, step, max_norm=0.5).cpu().numpy()
        norm, factor = grad_norm(list(g.values()), 0.5)
        assert factor < 1 and abs(clip[0] - norm) <= 2 * U * norm and abs(clip[1] - factor) <= 4 * U * factor
        states = tw.twell_adamw_states(opt) if bits == 8 else (opt.m, opt.v)
        for i, n in enumerate(block.NAMES):
            w, m, v = host[n]
            m, v = moments(m, v, g[n], 0.9, 0.999, clip[1])
            w = weights(w, m, v, 1e-2, step, 0.9, 0.999, 1e-8, 0.1 if i < 3 else 0.0)
            got = decode(from_dev(getattr(block, n), dtype), dtype).reshape(-1)
            kept = decode(from_dev(getattr(block, n), dtype), dtype).reshape(-1) if not master else opt.master[i].cpu().numpy().reshape(-1)
            bound = 1e-2 * 16 * U + 4 * U * np.abs(w)
            if master:
                assert (np.abs(kept - w) <= bound).all(), n
                assert_bitwise(from_dev(getattr(block, n), dtype).reshape(-1), round_to_storage(kept.astype(np.float64), dtype), n)
            else:
                # rounded to one of the two neighbours: less than one step of 2^-7
                assert (np.abs(got - w) <= 2.0 ** -7 * (np.abs(w) + bound) + bound).all(), n
            # what the next step starts from is what the GPU holds
            host[n] = [kept.astype(np.float64)] + [t[i].float().cpu().numpy().reshape(-1) for t in states]
        code, byte = unpack(block.mx4_gate.q.cpu().numpy(), block.mx4_gate.scale.cpu().numpy(), 512)
        want_code, want_byte = quantize(decode(from_dev(block.w_gate, dtype), dtype))
        assert_bitwise(code, want_code, "the gate's codes")
        assert_bitwise(byte, want_byte, "the gate's scales")
    y, _ = block.serve_mx4(dev["x"], dev["res"], dev["bias"])
    assert y.isfinite().all()


def test_serving_and_steps_under_graph_capture():
    """Two graphs, one workspace: captured once, replayed in turn with new inputs in the
    same buffers between eager work, every replay against the eager calls."""
    import torch
    T, d, F, dt = 300, 1024, 5000, torch.bfloat16
    g = torch.Generator(device="cuda:0")
    g.manual_seed(3)

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda:0") * scale).to(dt)

    x, res, w = rand(T, d), rand(T, d), torch.ones(d, device="cuda:0", dtype=dt)
    wg, wl = rand(F, d, scale=d ** -0.5), rand(200, 65536, scale=1 / 256)
    gate, long = tw.twell_quantize_mx4(wg), tw.twell_quantize_mx4(wl)
    xl = rand(T, 65536)
    assert tw.twell_mx4_matmul_workspace_size(T, 200, 65536) > 0  # ranges of K
    ws = torch.empty(max(tw.twell_mx4_matmul_workspace_size(T, F, d), tw.twell_mx4_matmul_workspace_size(T, 200, 65536),
                         1 << 16), dtype=torch.uint8, device="cuda:0")
    h, y = torch.empty_like(x), torch.empty_like(x)
    q, ql = tw.Mx4Rows.empty(T, d, "cuda:0", factor=True), tw.Mx4Rows.empty(T, 65536, "cuda:0")
    out, outl = torch.empty(T, F, dtype=dt, device="cuda:0"), torch.empty(T, 200, device="cuda:0")
    grads = [rand(F, d), torch.randn(d, generator=g, device="cuda:0")]
    opt = tw.TwellAdamW.zeros([wg, w], bits=8)
    clip = torch.empty(2, device="cuda:0")
    count = torch.zeros(1, dtype=torch.int64, device="cuda:0")

    def serve():
        tw.twell_rmsnorm_mx4(x, w, EPS, residual=res, h=h, y=y, q=q)
        tw.twell_mx4_matmul(q, gate, y=out, workspace=ws)
        tw.twell_quantize_mx4(xl, ql)
        tw.twell_mx4_matmul(ql, long, y=outl, workspace=ws)

    def train():
        count.add_(1)
        tw.twell_grad_norm(grads, 1.0, out=clip, workspace=ws)
        tw.twell_adamw_step(opt, grads, lr=1e-3, step=count, clip=clip)
        tw.twell_quantize_mx4(wg, gate)

    held = [wg, w, *opt.m, *opt.v, *opt.m_scale, *opt.v_scale, count]

    def both():
        serve()
        a = [t.clone() for t in (h, y, q.q, q.scale, q.factor, out, outl)]
        train()
        return a + [t.clone() for t in held + [clip, gate.q, gate.scale]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for f in (serve, train):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        graphs.append(graph)
    for i in range(4):
        x.copy_(rand(T, d))
        xl.copy_(rand(T, 65536))
        grads[0].copy_(rand(F, d))
        start = [t.clone() for t in held]
        torch.cuda.synchronize()
        graphs[0].replay()
        got = [t.clone() for t in (h, y, q.q, q.scale, q.factor, out, outl)]
        graphs[1].replay()
        got += [t.clone() for t in held + [clip, gate.q, gate.scale]]
        torch.cuda.synchronize()
        for t, b in zip(held, start):
            t.copy_(b)
        for t in (h, y, out, outl, clip):
            t.zero_()
        tw.twell_quantize_mx4(wg, gate)
        want = both()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (i, k)


def test_two_streams_at_once():
    import torch
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for i in range(2):
        g = torch.Generator(device="cuda:0")
        g.manual_seed(10 + i)
        x = torch.randn(200 + i, 40000, generator=g, device="cuda:0")
        w = torch.randn(300, 40000, generator=g, device="cuda:0")
        p = torch.randn(200000 + i, generator=g, device="cuda:0")
        sets.append((x, w, p, [torch.randn_like(p)]))

    def work(x, w, p, grads):
        opt = tw.TwellAdamW.zeros([p.clone()], bits=8)
        out = []
        for t in (1, 2, 3):
            y = tw.twell_mx4_matmul(tw.twell_quantize_mx4(x), tw.twell_quantize_mx4(w), dtype=torch.float32)
            tw.twell_adamw_step(opt, grads, lr=1e-3, step=t, clip=tw.twell_grad_norm(grads, 1.0))
            out.append(y)
        return out + [opt.weights[0], opt.m[0], opt.v[0]]

    want = [work(*s) for s in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for i, st in enumerate(streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got[i] = work(*sets[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_larger_buffer_keeps_what_lies_round_it():
    # outputs as row slices of larger buffers: the rows before and behind stay
    import torch
    for dt in (torch.bfloat16, torch.float32):
        x = torch.randn(40, 96, device="cuda:0").to(dt)
        buf = tw.Mx4Rows.empty(60, 96, "cuda:0", factor=True)
        for t in (buf.q, buf.scale):
            t.fill_(0xAB)
        buf.factor.fill_(7.0)
        part = tw.Mx4Rows(buf.q[10:50], buf.scale[10:50], 96, buf.factor[10:50])
        tw.twell_rmsnorm_mx4(x, torch.ones(96, device="cuda:0", dtype=dt), q=part)
        for t, fill in ((buf.q, 0xAB), (buf.scale, 0xAB), (buf.factor, 7.0)):
            assert (t[:10] == fill).all() and (t[50:] == fill).all()
        assert (buf.q[10:50] != 0xAB).any()
        assert (part.factor != 7.0).all()
