"""The feed-forward block of examples/ffn_block.py: serving with the gate in 8
bits and a training step, against the float64 oracle, and the block operators
under HIP graph capture."""

import importlib.util
import os

import numpy as np
import pytest

from oracle.block import int8_matmul, quantize_rows, residual_sum, rmsnorm, rmsnorm_backward, rmsnorm_quantized
from oracle.backward import ffn_backward
from oracle.ffn import ffn, ffn_from_h, rel_l2
from oracle.numerics import decode, round_to_storage
from oracle.twell import relu_storage
from workloads.synth import to_storage

from gpu_util import TOL, assert_bitwise, from_dev, to_dev, torch_dtype

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EPS = 1e-6


def _example():
    spec = importlib.util.spec_from_file_location("ffn_block", os.path.join(ROOT, "examples", "ffn_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _inputs(T, d, F, dtype, seed, density=0.02):
    from statistics import NormalDist
    rng = np.random.default_rng(seed)
    s = {k: to_storage(v, dtype) for k, v in {
        "x": rng.standard_normal((T, d)), "res": rng.standard_normal((T, d)),
        "norm": 1.0 + 0.1 * rng.standard_normal(d), "wg": rng.standard_normal((F, d)) / d ** 0.5,
        "wu": rng.standard_normal((F, d)) / d ** 0.5, "wd": rng.standard_normal((F, d)) / F ** 0.5,
        "dy": rng.standard_normal((T, d)), "dh": rng.standard_normal((T, d))}.items()}
    s["bias"] = np.full(T, NormalDist().inv_cdf(density), np.float32)
    return s


def _block(s, dtype, cap=32, tile=128):
    import torch
    ex = _example()
    dev = {k: to_dev(v, dtype) for k, v in s.items() if k != "bias"}
    dev["bias"] = torch.from_numpy(s["bias"]).to("cuda:0")
    return ex.FfnBlock(dev["norm"], dev["wg"], dev["wu"], dev["wd"], EPS, tile=tile, cap=cap), dev


@pytest.mark.parametrize("dtype,T,d,F", [("f32", 67, 256, 512), ("bf16", 96, 512, 1024), ("bf16", 1, 512, 1024)])
def test_serving_block(dtype, T, d, F):
    s = _inputs(T, d, F, dtype, 1)
    block, dev = _block(s, dtype)
    y, h = block.serve(dev["x"], dev["res"], dev["bias"])
    h_o = residual_sum(s["x"], s["res"], dtype)
    assert_bitwise(from_dev(h, dtype), h_o, "h")
    # the block from its definition: norm, its 8 bits, the product with the
    # weights' 8 bits, then the layer with those gate activations
    q, scale = rmsnorm_quantized(h_o, s["norm"], EPS, dtype)
    qw, sw = quantize_rows(s["wg"], dtype)
    pre = round_to_storage(int8_matmul(q, scale, qw, sw, s["bias"]), dtype)
    act = relu_storage(pre, dtype)
    n = round_to_storage(rmsnorm(h_o, s["norm"], EPS, dtype), dtype)
    want = ffn_from_h(decode(act, dtype), n, s["wu"], s["wd"], dtype)
    assert np.count_nonzero(decode(act, dtype) > 0, axis=1).max() > 0
    assert rel_l2(decode(from_dev(y, dtype), dtype), want) <= TOL[dtype]
    # the block whose gate is not in 8 bits
    y16, h16 = block.forward(dev["x"], dev["res"], dev["bias"])
    assert_bitwise(from_dev(h16, dtype), h_o, "h of the bf16 block")
    want16 = ffn(n, s["wg"], s["wu"], s["wd"], s["bias"], dtype)
    assert rel_l2(decode(from_dev(y16, dtype), dtype), want16) <= TOL[dtype]


@pytest.mark.parametrize("dtype,T,d,F", [("f32", 64, 256, 512), ("bf16", 96, 512, 1024)])
def test_training_step(dtype, T, d, F):
    s = _inputs(T, d, F, dtype, 2)
    block, dev = _block(s, dtype)
    lam = 2e-5
    y, h, grads = block.train_step(dev["x"], dev["res"], dev["dy"], dev["dh"], dev["bias"], lam, width=64)
    h_o = residual_sum(s["x"], s["res"], dtype)
    assert_bitwise(from_dev(h, dtype), h_o, "h")
    # The layer's oracle takes the normed rows and gate activations as the step
    # stored them (the same kernels give the same bits again): a last-bit
    # difference in a normed row could switch a unit whose gate is near zero.
    nd = tw.twell_rmsnorm(dev["x"], dev["norm"], EPS, residual=dev["res"]).y
    _, pre = tw.twell_gate_pack(nd, dev["wg"], dev["bias"], tile=128, cap=32, pre_out=True)
    n, act = from_dev(nd, dtype), relu_storage(from_dev(pre, dtype), dtype)
    ref = ffn_backward(n, s["wg"], s["wu"], s["wd"], act, s["dy"], float(np.float32(lam)), dtype)
    assert rel_l2(decode(from_dev(y, dtype), dtype), ffn_from_h(decode(act, dtype), n, s["wu"], s["wd"], dtype)) <= TOL[dtype]
    for k, r in (("w_gate", "dw_gate"), ("w_up", "dw_up"), ("w_down", "dw_down")):
        assert rel_l2(grads[k].cpu().numpy().astype(np.float64), ref[r]) <= 1e-5, k
    # the layer's dx carries its own tolerance; the norm is linear in it and
    # rounds once more
    dx, dnorm = rmsnorm_backward(round_to_storage(ref["dx"], dtype), h_o, s["norm"], EPS, dtype, s["dh"])
    assert rel_l2(decode(from_dev(grads["dx"], dtype), dtype), dx) <= 2 * TOL[dtype]
    assert rel_l2(grads["norm_weight"].cpu().numpy().astype(np.float64), dnorm) <= 2 * TOL[dtype]


def test_under_graph_capture():
    """Captured once, replayed with new inputs in the same buffers between eager work."""
    import torch
    T, d, F, dt = 48, 1024, 512, torch.bfloat16
    g = torch.Generator(device="cuda:0")
    g.manual_seed(3)
    x, res = (torch.randn(T, d, generator=g, device="cuda:0").to(dt) for _ in range(2))
    w = torch.ones(d, device="cuda:0", dtype=dt)
    qw, sw = tw.twell_quantize_rows(torch.randn(F, d, generator=g, device="cuda:0").to(dt))
    h, y = torch.empty_like(x), torch.empty_like(x)
    q, sc = torch.empty(T, d, dtype=torch.int8, device="cuda:0"), torch.empty(T, device="cuda:0")
    out = torch.empty(T, F, dtype=dt, device="cuda:0")
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda:0")
    ws = torch.empty(max(tw.twell_int8_matmul_workspace_size(T, F, d), 256), dtype=torch.uint8, device="cuda:0")
    wb = torch.empty(tw.twell_rmsnorm_backward_workspace_size(T, d, dt), dtype=torch.uint8, device="cuda:0")

    def step():
        tw.twell_rmsnorm(x, w, EPS, residual=res, h=h, y=y, q=q, scale=sc)
        tw.twell_int8_matmul(q, sc, qw, sw, y=out, workspace=ws)
        tw.twell_rmsnorm_backward(y, h, w, EPS, dh=x, dx=dx, dweight=dw, workspace=wb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn(T, d, generator=g, device="cuda:0"))
        res.copy_(torch.randn(T, d, generator=g, device="cuda:0"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, y, q, sc, out, dx, dw)]
        for t in (h, y, q, sc, out, dx, dw):
            t.zero_()
        step()
        torch.cuda.synchronize()
        for a, b, name in zip(got, (h, y, q, sc, out, dx, dw), ("h", "y", "q", "scale", "out", "dx", "dweight")):
            assert torch.equal(a, b), (i, name)
