"""Cases of the block operators around the feed-forward layer: the residual
RMS norm and its gradient, the 8-bit row quantiser and the 8-bit matrix
product.

``run`` computes each operator in plain torch operations (32-bit floats, one
rounding at the end) or, with ``own`` set, through the library's entry points.
Definitions, for rows t of length d:

    h = round(x + residual)                      (residual stream, storage type)
    r_t = 1 / sqrt(mean_j h_tj^2 + eps),  y_tj = round(h_tj * r_t * w_j)
    8 bits: z = h * w, m_t = max(max_j |z_tj|, 2^-100),
            q_tj = rint(z_tj * (127 / m_t)),  scale_t = r_t * (m_t / 127)
    gradient: g = dy * w,  dx = round(dh + r * (g - h * r^2 * mean(g * h))),
              dw_j = sum_t dy_tj * h_tj * r_t
    quantiser: as the 8 bits above with z = x and r = 1
    product: y_mn = round((sum_k a_mk b_nk) * sa_m * sb_n + bias_m)

What is held in 8 bits is returned as the values that it stands for, in the
activations' type.
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
QMAX = 127.0
TINY = 2.0 ** -100
DEVICE = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # decoding: one new token enters the block
        {"name": "norm one token", "op": "norm", "T": 1, "d": 2048, "dtype": "bf16", "residual": True, "quantize": False},
        # a batch of four 2048-token prompts through the 1.5B-class layer, with
        # the 8-bit copy for the gate's product beside y for the gathers
        {"name": "norm prompts", "op": "norm", "T": 8192, "d": 2048, "dtype": "bf16", "residual": True, "quantize": True},
        # an odd batch in fp32, rows that are not whole 64-lane vectors
        {"name": "norm ragged", "op": "norm", "T": 1999, "d": 1000, "dtype": "f32", "residual": True, "quantize": True},
        # training the 1.5B-class layer: gradient through the norm, joined with
        # the gradient that arrives along the residual stream
        {"name": "norm gradient", "op": "norm_grad", "T": 8192, "d": 2048, "dtype": "bf16", "stream": True},
        # a short odd fp32 batch
        {"name": "norm gradient ragged", "op": "norm_grad", "T": 67, "d": 1000, "dtype": "f32", "stream": False},
        # the hidden activations of the 1.5B-class layer before an 8-bit down product
        {"name": "quantise activations", "op": "quantize", "rows": 8192, "cols": 8192, "dtype": "bf16"},
        # a small odd fp32 matrix
        {"name": "quantise ragged", "op": "quantize", "rows": 130, "cols": 1000, "dtype": "f32"},
        # decoding: one token through a 1.5B-class gate
        {"name": "product one token", "op": "product", "M": 1, "N": 8192, "K": 2048, "dtype": "bf16", "bias": False},
        # decoding: a batch of 64 tokens through the down projection
        {"name": "product 64 tokens", "op": "product", "M": 64, "N": 2048, "K": 8192, "dtype": "bf16", "bias": False},
        # the gate of the 1.5B-class layer on the whole batch, with the per-token bias
        {"name": "product prompts", "op": "product", "M": 8192, "N": 8192, "K": 2048, "dtype": "bf16", "bias": True},
        # the gate of the larger layer
        {"name": "product larger", "op": "product", "M": 16384, "N": 14336, "K": 4096, "dtype": "bf16", "bias": False},
        # odd sizes, fp32 results
        {"name": "product ragged", "op": "product", "M": 333, "N": 1000, "K": 777, "dtype": "f32", "bias": True},
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of [low, high]; every second one a multiple of 64 where it can be."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and n >= 64:
        n = n // 64 * 64
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "product", "product"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        d = _size(rng, 128, 8192)
        T = _size(rng, 1, min(16384, 8192 * 2048 // d))
        return {"op": op, "T": T, "d": d, "dtype": dtype, "residual": rng.random() < 0.7, "quantize": rng.random() < 0.5}
    if op == "norm_grad":
        d = _size(rng, 128, 8192)
        T = _size(rng, 1, min(16384, 8192 * 2048 // d))
        return {"op": op, "T": T, "d": d, "dtype": dtype, "stream": rng.random() < 0.7}
    if op == "quantize":
        cols = _size(rng, 128, 16384)
        return {"op": op, "rows": _size(rng, 1, min(16384, 8192 * 8192 // cols)), "cols": cols, "dtype": dtype}
    K = _size(rng, 256, 14336)
    N = _size(rng, 256, 14336)
    M = _size(rng, 1, 16384)
    M = min(M, 16384 * 14336 * 4096 // (N * K))
    return {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "bias": rng.random() < 0.5}


def _ceil16(n):
    return (n + 15) // 16 * 16


def _stream_rows(g, T, d, dtype):
    """Rows as a residual stream holds them: unequal tokens, and a few channels far larger than the rest."""
    v = torch.randn(T, d, generator=g, device=DEVICE)
    channel = torch.exp(0.5 * torch.randn(d, generator=g, device=DEVICE))
    channel[torch.randint(0, d, (max(1, d // 256),), generator=g, device=DEVICE)] *= 12.0
    token = torch.exp(0.3 * torch.randn(T, 1, generator=g, device=DEVICE))
    return (v * channel * token).to(TYPES[dtype])


def _int8_rows(g, rows, cols):
    """8-bit rows, 16-byte aligned as the quantiser lays them out, with scales of the usual size."""
    v = torch.randn(rows, _ceil16(cols), generator=g, device=DEVICE)
    v[:, cols:] = 0.0
    m = v.abs().amax(1, keepdim=True)
    q = torch.round(v * (QMAX / m)).to(torch.int8)
    return q[:, :cols], (m[:, 0] / QMAX).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "norm":
        T, d = case["T"], case["d"]
        s["x"] = _stream_rows(g, T, d, case["dtype"])
        s["residual"] = _stream_rows(g, T, d, case["dtype"]) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEVICE)).to(TYPES[case["dtype"]])
    elif op == "norm_grad":
        T, d = case["T"], case["d"]
        s["h"] = _stream_rows(g, T, d, case["dtype"])
        s["weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEVICE)).to(TYPES[case["dtype"]])
        s["dy"] = torch.randn(T, d, generator=g, device=DEVICE).to(TYPES[case["dtype"]])
        s["dh"] = torch.randn(T, d, generator=g, device=DEVICE).to(TYPES[case["dtype"]]) if case["stream"] else None
    elif op == "quantize":
        s["x"] = _stream_rows(g, case["rows"], case["cols"], case["dtype"])
    else:
        s["a"], s["a_scale"] = _int8_rows(g, case["M"], case["K"])
        s["b"], s["b_scale"] = _int8_rows(g, case["N"], case["K"])
        s["b_scale"] /= math.sqrt(case["K"])
        s["bias"] = torch.randn(case["M"], generator=g, device=DEVICE) - 2.3 if case["bias"] else None
    return s


# ---- plain form -------------------------------------------------------------

def _quantized(z, r, dtype):
    # whole tensors on both sides of each division: torch divides by or into a
    # Python number through a rounded reciprocal, which moves values near a tie
    m = z.abs().amax(1, keepdim=True).clamp_min(TINY)
    top = torch.full_like(m, QMAX)
    return (torch.round(z * (top / m)) * (r * (m / top))).to(dtype)


def _plain_norm(s):
    dtype = s["x"].dtype
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dtype)
    hf, w = h.float(), s["weight"].float()
    r = torch.rsqrt((hf * hf).mean(1, keepdim=True) + EPS)
    out = {"y": (hf * r * w).to(dtype)}
    if s["residual"] is not None:
        out["h"] = h
    if s["case"]["quantize"]:
        out["q"] = _quantized(hf * w, r, dtype)
    return out


def _plain_norm_grad(s):
    h, dy, w = s["h"].float(), s["dy"].float(), s["weight"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    g = dy * w
    dx = r * (g - h * (r * r * (g * h).mean(1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * h * r).sum(0)}


def _plain_product(s):
    y = torch.matmul(s["a"].float(), s["b"].float().t())
    y = y * s["a_scale"][:, None] * s["b_scale"]
    if s["bias"] is not None:
        y = y + s["bias"][:, None]
    return y.to(TYPES[s["case"]["dtype"]])


# ---- the library's operators --------------------------------------------------

def _values(q, scale, dtype):
    out = torch.empty(q.shape, dtype=dtype, device=q.device)
    return torch.mul(q, scale[:, None], out=out)


def _own_run(s):
    import activation_sparse_transformer_bf16_amd as tw

    op = s["case"]["op"]
    if op == "norm":
        n = tw.twell_rmsnorm(s["x"], s["weight"], eps=EPS, residual=s["residual"], quantize=s["case"]["quantize"])
        out = {"y": n.y}
        if s["residual"] is not None:
            out["h"] = n.h
        if s["case"]["quantize"]:
            out["q"] = _values(n.q, n.scale, s["x"].dtype)
        return out
    if op == "norm_grad":
        dx, dweight = tw.twell_rmsnorm_backward(s["dy"], s["h"], s["weight"], eps=EPS, dh=s["dh"])
        return {"dx": dx, "dweight": dweight}
    if op == "quantize":
        q, scale = tw.twell_quantize_rows(s["x"])
        return _values(q, scale, s["x"].dtype)
    return tw.twell_int8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], row_bias=s["bias"],
                                dtype=TYPES[s["case"]["dtype"]])


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_grad":
        return _plain_norm_grad(state)
    if op == "quantize":
        x = state["x"].float()
        return _quantized(x, 1.0, state["x"].dtype)
    return _plain_product(state)


def work(case):
    op = case["op"]
    s = 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        n, d = case["T"] * case["d"], case["d"]
        moved = n * s * (4 if case["residual"] else 2) + d * s  # x, residual, h and y; the weight
        flops = 4 * n
        if case["quantize"]:
            moved += n * s  # the values returned for the 8 bits
            flops += 4 * n
        return {"bytes": moved, "flops": flops}
    if op == "norm_grad":
        n, d = case["T"] * case["d"], case["d"]
        return {"bytes": n * s * (4 if case["stream"] else 3) + d * (s + 4), "flops": 12 * n}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * s, "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": M * K + N * K + M * N * s + 4 * (M + N + (M if case["bias"] else 0)), "flops": 2 * M * N * K}


# ---- 64 bits --------------------------------------------------------------------

def _exact_quantized(z, factor):
    """The quantiser's values in 64 bits: z rows onto 255 levels of their largest magnitude, times factor."""
    top = torch.maximum(z.abs().max(dim=1).values, torch.full((), TINY, dtype=torch.float64, device=z.device))
    step = (top / 127).unsqueeze(1)
    return torch.round(z / step) * step * factor


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        w = s["weight"].double()
        root = (h.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS).sqrt()
        out = {"y": h / root * w}
        if s["residual"] is not None:
            out["h"] = h
        if case["quantize"]:
            out["q"] = _exact_quantized(h * w, 1.0 / root)
        return out
    if op == "norm_grad":
        # d/dh of w h / root: dy w / root - h (dy w . h) / (d root^3)
        h, dy, w = s["h"].double(), s["dy"].double(), s["weight"].double()
        root = (h.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS).sqrt()
        dot = (dy * w * h).sum(dim=1, keepdim=True)
        dx = dy * w / root - h * dot / (case["d"] * root ** 3)
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dweight": (dy * h / root).sum(dim=0)}
    if op == "quantize":
        return _exact_quantized(s["x"].double(), 1.0)
    # products of 8-bit integers are exact in 64-bit floats
    a = s["a"].double() * s["a_scale"].double()[:, None]
    b = s["b"].double() * s["b_scale"].double()[:, None]
    y = a.mm(b.t().contiguous())
    return y if s["bias"] is None else y + s["bias"].double()[:, None]
