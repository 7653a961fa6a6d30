"""A pre-norm feed-forward block: residual addition, RMS norm, sparse ReLU-gated
FFN -- serving with the gate in 8 or 4 bits, and training steps through the norm.

    python examples/ffn_block.py [--tokens 8192] [--d-model 2048] [--d-ff 8192]

Serving runs twell_rmsnorm (which writes the normed rows in bf16 and in 8 bits),
twell_int8_matmul with the gate's 8-bit weights, twell_pack of the gate's
pre-activations and twell_sparse_ffn; with the gate in 4 bits the first two are
twell_rmsnorm_mx4 and twell_mx4_matmul; the bf16 block runs twell_rmsnorm and
twell_ffn_forward.  Rows that overflow the TwELL capacity take the dense
fallback, which computes their gate from the bf16 weights.  Training keeps h and
the activations and goes back through twell_ffn_backward and
twell_rmsnorm_backward; twell_grad_norm and twell_adamw_step then update the block's
weights, and the gate's narrow copies are made anew.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import activation_sparse_transformer_bf16_amd as tw  # noqa: E402


class FfnBlock:
    """Weights of one block ([F, d] rows as the library takes them), the gate's 8-bit and 4-bit copies beside them."""

    def __init__(self, norm_weight, w_gate, w_up, w_down, eps: float = 1e-6, tile: int = 256, cap: int = 16):
        self.norm_weight, self.w_gate, self.w_up, self.w_down = norm_weight, w_gate, w_up, w_down
        self.eps, self.tile, self.cap = eps, tile, cap
        self.q_gate, self.gate_scale = tw.twell_quantize_rows(w_gate)  # once, at load time
        self.mx4_gate = tw.twell_quantize_mx4(w_gate)

    def serve(self, x, residual, gate_bias=None):
        """(y, h): the block's output and the updated residual stream; the gate in 8 bits."""
        n = tw.twell_rmsnorm(x, self.norm_weight, self.eps, residual=residual, quantize=True)
        pre = tw.twell_int8_matmul(n.q, n.scale, self.q_gate, self.gate_scale, row_bias=gate_bias, dtype=x.dtype)
        packed = tw.twell_pack(pre, self.tile, self.cap, dense=False)
        y = tw.twell_sparse_ffn(packed, n.y, self.w_gate, self.w_up, self.w_down, gate_bias)
        return y, n.h

    def serve_mx4(self, x, residual, gate_bias=None):
        """The same with the gate in 4 bits."""
        n = tw.twell_rmsnorm_mx4(x, self.norm_weight, self.eps, residual=residual)
        pre = tw.twell_mx4_matmul(n.q, self.mx4_gate, row_bias=gate_bias, dtype=x.dtype)
        packed = tw.twell_pack(pre, self.tile, self.cap, dense=False)
        y = tw.twell_sparse_ffn(packed, n.y, self.w_gate, self.w_up, self.w_down, gate_bias)
        return y, n.h

    def forward(self, x, residual, gate_bias=None):
        """The same block with the gate in the activations' type."""
        n = tw.twell_rmsnorm(x, self.norm_weight, self.eps, residual=residual)
        y, _ = tw.twell_ffn_forward(n.y, self.w_gate, self.w_up, self.w_down, gate_bias, self.tile, self.cap)
        return y, n.h

    def train_step(self, x, residual, dy, dh, gate_bias=None, lam: float = 0.0, width: int = 256):
        """Forward and backward: (y, h, gradients) for the gradients dy of y and dh
        of h; ``dx`` is the gradient of x and of the residual alike."""
        n = tw.twell_rmsnorm(x, self.norm_weight, self.eps, residual=residual)
        packed = tw.TwellMatrix.empty(x.shape[0], self.w_gate.shape[0], self.tile, self.cap, x.dtype, x.device, u=True)
        y, _ = tw.twell_ffn_forward(n.y, self.w_gate, self.w_up, self.w_down, gate_bias, packed=packed)
        hybrid = tw.twell_to_hybrid(packed, width)
        dn, dw_gate, dw_up, dw_down = tw.twell_ffn_backward(hybrid, n.y, self.w_gate, self.w_up, self.w_down, dy, lam)
        dx, dnorm = tw.twell_rmsnorm_backward(dn, n.h, self.norm_weight, self.eps, dh=dh)
        return y, n.h, {"dx": dx, "norm_weight": dnorm, "w_gate": dw_gate, "w_up": dw_up, "w_down": dw_down}

    NAMES = ("w_gate", "w_up", "w_down", "norm_weight")

    def optimizer(self, bits: int = 8, master: bool = False, weight_decay: float = 0.1) -> tw.TwellAdamW:
        """AdamW's states for the block's weights, before the first step (the norm's weight without decay)."""
        return tw.TwellAdamW.zeros([getattr(self, n) for n in self.NAMES], bits, master, [weight_decay] * 3 + [0.0])

    def update(self, opt: tw.TwellAdamW, grads, lr: float, step: int, max_norm: float = 1.0):
        """One optimiser step with train_step()'s gradients, clipped to max_norm
        together; returns their norm and the factor.  The gate's narrow copies follow."""
        g = [grads[n] for n in self.NAMES]
        clip = tw.twell_grad_norm(g, max_norm)
        tw.twell_adamw_step(opt, g, lr=lr, step=step, clip=clip)
        tw.twell_quantize_rows(self.w_gate, self.q_gate, self.gate_scale)
        tw.twell_quantize_mx4(self.w_gate, self.mx4_gate)
        return clip


def _time(f, n: int = 20) -> float:
    """Microseconds a call, back to back."""
    for _ in range(5):
        f()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n * 1e3


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--d-model", type=int, default=2048)
    ap.add_argument("--d-ff", type=int, default=8192)
    ap.add_argument("--density", type=float, default=0.01, help="active gate units per token")
    a = ap.parse_args()
    from statistics import NormalDist

    T, d, F = a.tokens, a.d_model, a.d_ff
    g = torch.Generator(device="cuda:0")
    g.manual_seed(0)

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda:0") * scale).bfloat16()

    block = FfnBlock((1.0 + 0.1 * torch.randn(d, generator=g, device="cuda:0")).bfloat16(),
                     rand(F, d, scale=d ** -0.5), rand(F, d, scale=d ** -0.5), rand(F, d, scale=F ** -0.5))
    x, residual = rand(T, d), rand(T, d)
    bias = torch.full((T,), NormalDist().inv_cdf(a.density), device="cuda:0")
    y8, h8 = block.serve(x, residual, bias)
    y16, h16 = block.forward(x, residual, bias)
    y4, h4 = block.serve_mx4(x, residual, bias)
    for bits, y, h in ((8, y8, h8), (4, y4, h4)):
        far = float((y.float() - y16.float()).norm() / y16.float().norm())
        print(f"{T} tokens, {d} x {F}: {bits}-bit gate against bf16 gate: y differs by {far:.3f} of its norm, "
              f"h {'equal' if torch.equal(h, h16) else 'DIFFERENT'}")
    print(f"serving, gate in 8 bits {_time(lambda: block.serve(x, residual, bias)):8.1f} us")
    print(f"serving, gate in 4 bits {_time(lambda: block.serve_mx4(x, residual, bias)):8.1f} us")
    print(f"serving, gate in bf16   {_time(lambda: block.forward(x, residual, bias)):8.1f} us")
    dy, dh = rand(T, d, scale=0.1), rand(T, d, scale=0.1)
    print(f"training step           {_time(lambda: block.train_step(x, residual, dy, dh, bias), 10):8.1f} us")
    grads = block.train_step(x, residual, dy, dh, bias)[2]
    for bits, master in ((32, True), (8, False)):
        opt, steps = block.optimizer(bits, master), iter(range(1, 100))
        print(f"AdamW, {bits}-bit states{', fp32 copies' if master else ''}: "
              f"{_time(lambda: block.update(opt, grads, 1e-4, next(steps)), 10):8.1f} us")


if __name__ == "__main__":
    main()
