"""Cases of the microscaled operators: rows of 4-bit floats (their quantiser,
the norm that writes them, their product) and the AdamW step over many tensors,
with states in 32 bits or in microscaled 8 bits and gradients clipped by their
norm.

``run`` computes each operator in plain torch operations or, with ``own`` set,
through the library's entry points.  Definitions:

    4 bits: blocks of 32 along a row share a scale 2^e, e the smallest whole
            number (-126 ... 126) with max |z| <= 7 * 2^e; an element is the
            nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code) times
            2^e with z's sign.  A byte holds two elements, the even one low.
            Scale bytes are e + 127; block b of a row is byte
            16 * (b / 16) + 4 * (b % 4) + b / 4 % 4.
    norm:   h = round(x + residual), r_t = 1 / sqrt(mean_j h_tj^2 + eps),
            y = round(h r w); the 4 bits are those of z = h w (rounded to fp32)
            and stand for themselves times r_t
    product: y_mn = round(sum_k a_mk b_nk + bias_m)
    clip:   norm = sqrt(sum of all gradients' squares), factor = min(1, max / norm)
    step:   g = grad * factor,  m = b1 m + (1 - b1) g,  v = b2 v + ((1 - b2) g) g,
            w = (1 - lr decay) w - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps)
    8 bits: blocks of 32 of a tensor share 2^E, E the smallest whole number
            (-87 ... 113) with max <= 1.875 * 2^E; m is a sign, 4 exponent and 3
            mantissa bits, v 5 and 3, both with subnormals and the topmost
            exponent standing for 2^E; rounded down where the part cut off plus a
            dither in (0, 1) stays below one step, up otherwise; v > 0 is not
            rounded to 0.  Scale bytes are E + 127.
    bf16 weights without an fp32 copy are rounded by a dither in the same way.
    dither: a hash of the step, the tensor's place in the list and the element
            (``_random``).

What is held in 4 or 8 bits is returned as the values that it stands for, 4 bits
in the activations' type and 8 bits in bf16 (which holds them exactly).
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
DEVICE = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LR, BETA1, BETA2, ADAM_EPS, DECAY, MAX_NORM = 1e-3, 0.9, 0.95, 1e-8, 0.1, 1.0


def listed():
    return [
        # the hidden activations of the 1.5B-class layer before a 4-bit down product
        {"name": "quantise activations", "op": "quantize", "rows": 8192, "cols": 8192, "dtype": "bf16"},
        # a small odd fp32 matrix
        {"name": "quantise ragged", "op": "quantize", "rows": 130, "cols": 1000, "dtype": "f32"},
        # decoding: one new token enters the block, its 4 bits go to the gate's product
        {"name": "norm one token", "op": "norm", "T": 1, "d": 2048, "dtype": "bf16", "residual": True},
        # a batch of four 2048-token prompts through the 1.5B-class layer
        {"name": "norm prompts", "op": "norm", "T": 8192, "d": 2048, "dtype": "bf16", "residual": True},
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
        # training the 1.5B-class layer: three matrices and the norm's weight, fp32
        # copies of the bf16 weights, fp32 states and gradients
        {"name": "step layer", "op": "step", "matrices": 3, "n": 8192 * 2048, "vectors": 1, "d": 2048,
         "dtype": "bf16", "master": True, "bits": 32, "grad": "f32", "clip": True},
        # the same in little memory: bf16 weights alone, states in 8 bits
        {"name": "step layer 8 bits", "op": "step", "matrices": 3, "n": 8192 * 2048, "vectors": 1, "d": 2048,
         "dtype": "bf16", "master": False, "bits": 8, "grad": "f32", "clip": True},
        # many small odd tensors of an fp32 model
        {"name": "step ragged 8 bits", "op": "step", "matrices": 5, "n": 130 * 333, "vectors": 8, "d": 333,
         "dtype": "f32", "master": False, "bits": 8, "grad": "f32", "clip": True},
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of [low, high]; every second one a multiple of 64 where it can be."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and n >= 64:
        n = n // 64 * 64
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["quantize", "norm", "product", "product", "step", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "quantize":
        cols = _size(rng, 128, 16384)
        return {"op": op, "rows": _size(rng, 1, min(16384, 8192 * 8192 // cols)), "cols": cols, "dtype": dtype}
    if op == "norm":
        d = _size(rng, 128, 8192)
        T = _size(rng, 1, min(16384, 8192 * 2048 // d))
        return {"op": op, "T": T, "d": d, "dtype": dtype, "residual": rng.random() < 0.7}
    if op == "product":
        K = _size(rng, 256, 14336)
        N = _size(rng, 256, 14336)
        M = min(_size(rng, 1, 16384), 16384 * 14336 * 4096 // (N * K))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "bias": rng.random() < 0.5}
    matrices = rng.randint(1, 6)
    return {"op": op, "matrices": matrices, "n": _size(rng, 1000, 3 * 8192 * 2048 // matrices),
            "vectors": rng.randint(0, 8), "d": _size(rng, 1, 8192), "dtype": dtype,
            "master": dtype == "bf16" and rng.random() < 0.5, "bits": rng.choice([8, 32]),
            "grad": rng.choice(["bf16", "f32"]), "clip": rng.random() < 0.7}


# ---- inputs -----------------------------------------------------------------------

def _ceil(n, k):
    return (n + k - 1) // k * k


def _stream_rows(g, T, d, dtype):
    """Rows as a residual stream holds them: unequal tokens, and a few channels far larger than the rest."""
    v = torch.randn(T, d, generator=g, device=DEVICE)
    channel = torch.exp(0.5 * torch.randn(d, generator=g, device=DEVICE))
    channel[torch.randint(0, d, (max(1, d // 256),), generator=g, device=DEVICE)] *= 12.0
    token = torch.exp(0.3 * torch.randn(T, 1, generator=g, device=DEVICE))
    return (v * channel * token).to(TYPES[dtype])


def _mx4_rows(g, rows, cols, size):
    """Rows in 4 bits as the quantiser lays them out: q [rows, cols / 2], 16-byte aligned rows, and scales
    [rows, a multiple of 16]; what lies behind a row's end is arbitrary."""
    z = torch.randn(rows, _ceil(cols, 32), generator=g, device=DEVICE) * size
    z[:, cols:] = 0.0
    code, byte = _mx4_codes(z)
    ld, lds = _ceil((cols + 1) // 2, 16), _ceil(_ceil(cols, 32) // 32, 16)
    q = torch.randint(0, 256, (rows, ld), generator=g, device=DEVICE, dtype=torch.uint8)
    pairs = code.view(rows, -1, 2)
    n = (cols + 1) // 2
    q[:, :n] = (pairs[:, :n, 0] | (pairs[:, :n, 1] << 4)).to(torch.uint8)
    scale = torch.randint(0, 256, (rows, lds), generator=g, device=DEVICE, dtype=torch.uint8)
    scale[:, _mx4_places(byte.shape[1])] = byte.to(torch.uint8)
    return q[:, :n], scale


def _mx4_places(blocks):
    b = torch.arange(blocks, device=DEVICE)
    return b // 16 * 16 + b % 4 * 4 + b // 4 % 4


def _sizes(case):
    return [case["n"]] * case["matrices"] + [case["d"]] * case["vectors"]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "quantize":
        s["x"] = _stream_rows(g, case["rows"], case["cols"], case["dtype"])
    elif op == "norm":
        T, d = case["T"], case["d"]
        s["x"] = _stream_rows(g, T, d, case["dtype"])
        s["residual"] = _stream_rows(g, T, d, case["dtype"]) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEVICE)).to(TYPES[case["dtype"]])
    elif op == "product":
        s["a"] = _mx4_rows(g, case["M"], case["K"], 1.0)
        s["b"] = _mx4_rows(g, case["N"], case["K"], 1.0 / math.sqrt(case["K"]))
        s["bias"] = torch.randn(case["M"], generator=g, device=DEVICE) - 2.3 if case["bias"] else None
    else:
        # a training run some way in: gradients of unequal size, states to match
        s["step"] = 1000
        s["weights"], s["master"], s["grads"], s["m"], s["v"], s["m_scale"], s["v_scale"] = [], [], [], [], [], [], []
        for n in _sizes(case):
            w = 0.02 * torch.randn(n, generator=g, device=DEVICE)
            size = 1e-3 * torch.exp(torch.randn(_ceil(n, 64) // 64, 1, generator=g, device=DEVICE))
            size = size.expand(-1, 64).reshape(-1)[:n]
            s["weights"].append(w.to(TYPES[case["dtype"]]))
            s["master"].append(w if case["master"] else None)
            s["grads"].append((size * torch.randn(n, generator=g, device=DEVICE)).to(TYPES[case["grad"]]))
            m = 0.2 * size * torch.randn(n, generator=g, device=DEVICE)
            v = size * size * torch.exp(0.5 * torch.randn(n, generator=g, device=DEVICE))
            ms = vs = None
            if case["bits"] == 8:
                m, ms = _state_codes(m, torch.full((n,), 0x8000, device=DEVICE, dtype=torch.int64), True)
                v, vs = _state_codes(v, torch.full((n,), 0x8000, device=DEVICE, dtype=torch.int64), False)
            s["m"].append(m)
            s["v"].append(v)
            s["m_scale"].append(ms)
            s["v_scale"].append(vs)
    return s


# ---- plain form -------------------------------------------------------------------

def _power(byte):
    """2^(byte - 127) for whole bytes of 1 to 254."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _power64(k):
    return ((k.long() + 1023) << 52).view(torch.float64)


def _mx4_round(z):
    """(level times sign, scale byte) of rows z whose length is a multiple of 32, in blocks [rows, blocks, 32]."""
    z = z.view(z.shape[0], -1, 32)
    top = z.abs().amax(2, keepdim=True)
    # the exponent, one higher where the mantissa is over 1.75
    byte = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 2).clamp(1, 253)
    a = z * _power(254 - byte)
    step = torch.where(a.abs() < 2.0, 0.5, torch.where(a.abs() < 4.0, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(-6.0, 6.0), byte


def _mx4_values(z, dtype, factor=None):
    """The values that z's 4 bits stand for, times factor, in dtype."""
    cols = z.shape[1]
    q, byte = _mx4_round(torch.nn.functional.pad(z, (0, -cols % 32)))
    out = (q * _power(byte)).view(z.shape[0], -1)[:, :cols]
    return (out if factor is None else out * factor).to(dtype)


def _mx4_codes(z):
    """(codes [rows, cols], scale bytes [rows, blocks]) of rows z whose length is a multiple of 32."""
    q, byte = _mx4_round(z)
    a = q.abs()
    code = torch.where(a <= 2.0, a * 2.0, torch.where(a <= 4.0, a + 2.0, a / 2.0 + 4.0)).to(torch.int32)
    return (code | ((z.view(q.shape) < 0).to(torch.int32) << 3)).view(z.shape[0], -1), byte[:, :, 0]


def _mx4_read(rows, cols):
    """The values of 4-bit rows, in fp32."""
    q, scale = rows
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=DEVICE)
    code = torch.stack((q & 15, q >> 4), 2).view(q.shape[0], -1)[:, :cols]
    blocks = _ceil(cols, 32) // 32
    size = _power(scale[:, _mx4_places(blocks)])
    return levels[code.int()] * size.repeat_interleave(32, 1)[:, :cols]


def _plain_norm(s):
    dtype = s["x"].dtype
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dtype)
    hf, w = h.float(), s["weight"].float()
    r = torch.rsqrt((hf * hf).mean(1, keepdim=True) + EPS)
    out = {"y": (hf * r * w).to(dtype), "q": _mx4_values(hf * w, dtype, r)}
    if s["residual"] is not None:
        out["h"] = h
    return out


def _plain_product(s):
    K = s["case"]["K"]
    y = torch.matmul(_mx4_read(s["a"], K), _mx4_read(s["b"], K).t())
    if s["bias"] is not None:
        y = y + s["bias"][:, None]
    return y.to(TYPES[s["case"]["dtype"]])


def _mix(x):
    """A 32-bit hash of whole numbers below 2^32 (an int64 tensor or a number)."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x85EBCA6B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(seed, place, n):
    """32 random bits for each element of the list's tensor `place`: m takes the low 16, v the high 16, a weight the middle ones."""
    key = _mix((_mix(seed) + place) & 0xFFFFFFFF)
    i = torch.arange(n, device=DEVICE)
    group = _mix(((i >> 3) + key) & 0xFFFFFFFF)
    x = ((group + (i & 7) * 0x9E3779B9) * 0x85EBCA6B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _state_codes(x, dither, signed):
    """x [n] in microscaled 8 bits: (codes, scale bytes), rounded by 16 bits of dither."""
    n = x.shape[0]
    a = torch.nn.functional.pad(x.abs(), (0, -n % 32)).view(-1, 32)
    dither = torch.nn.functional.pad(dither, (0, -n % 32)).view(-1, 32)
    byte = ((a.amax(1, keepdim=True).view(torch.int32) + 0xFFFFF) >> 23).clamp(40, 240)
    top = 15 if signed else 31
    # in 64 bits, where the part cut off is whole: v = fraction * 2^exponent
    v = a.double() * _power64(127 + top - 1 - byte)  # the smallest normal number is 1
    exponent = (torch.frexp(v)[1] - 1).clamp_min(0)
    part = torch.floor(v * _power64(3 - exponent) + (dither.double() + 0.5) / 65536.0).long()
    code = exponent * 8 + part  # a part of 8 ... 15 is a normal number of field exponent + 1
    if signed:
        code = code | ((torch.nn.functional.pad(x, (0, -n % 32)).view(-1, 32) < 0).long() << 7)
    else:
        code = torch.maximum(code, (a > 0).long())
    return code.view(-1)[:n].to(torch.uint8), byte.view(-1).to(torch.uint8)


def _state_read(code, byte, signed):
    """The values of microscaled 8-bit states, in fp32."""
    n = code.shape[0]
    c = code.int() & 127 if signed else code.int()
    field = (c >> 3).clamp_min(1)
    part = torch.where(c < 8, c, (c & 7) + 8).float()
    size = (byte.int().repeat_interleave(32)[:n] - (15 if signed else 31) + field - 3) << 23
    v = part * size.view(torch.float32)
    return torch.where(code > 127, -v, v) if signed else v


def _plain_clip(grads):
    total = torch.stack([g.double().square().sum() for g in grads]).sum()
    norm = total.sqrt().float()
    return torch.stack((norm, torch.clamp(torch.full_like(norm, MAX_NORM) / norm, max=1.0)))


def _plain_tensor(s, i, factor, t):
    """One tensor's step, in place."""
    c = s["case"]
    w, master, n = s["weights"][i], s["master"][i], s["weights"][i].shape[0]
    eight = c["bits"] == 8
    m = _state_read(s["m"][i], s["m_scale"][i], True) if eight else s["m"][i]
    v = _state_read(s["v"][i], s["v_scale"][i], False) if eight else s["v"][i]
    g = s["grads"][i].float()
    if factor is not None:
        g = g * factor
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * (1.0 - BETA2)) * g
    denom = torch.sqrt(v) / math.sqrt(1.0 - BETA2 ** t) + ADAM_EPS
    new = (w.float() if master is None else master) * (1.0 - LR * DECAY) - (LR / (1.0 - BETA1 ** t)) * (m / denom)
    bits = None
    if eight or (master is None and w.dtype == torch.bfloat16):
        bits = _random(t, i, n)
    if eight:
        code, byte = _state_codes(m, bits & 0xFFFF, True)
        s["m"][i].copy_(code)
        s["m_scale"][i].copy_(byte)
        code, byte = _state_codes(v, bits >> 16, False)
        s["v"][i].copy_(code)
        s["v_scale"][i].copy_(byte)
    else:
        s["m"][i].copy_(m)
        s["v"][i].copy_(v)
    if master is not None:
        master.copy_(new)
    elif w.dtype == torch.bfloat16:
        new = ((new.view(torch.int32) + ((bits >> 8) & 0xFFFF).int()) & -65536).view(torch.float32)
    w.copy_(new)
    out = {"w": w, "m": s["m"][i], "v": s["v"][i]}
    if eight:
        out["m"] = _state_read(s["m"][i], s["m_scale"][i], True).to(torch.bfloat16)
        out["v"] = _state_read(s["v"][i], s["v_scale"][i], False).to(torch.bfloat16)
    if master is not None:
        out["master"] = master
    return out


def _plain_step(s):
    clip = _plain_clip(s["grads"]) if s["case"]["clip"] else None
    s["step"] += 1
    out = [_plain_tensor(s, i, None if clip is None else clip[1], s["step"]) for i in range(len(s["grads"]))]
    return out if clip is None else out + [clip]


# ---- the library's operators --------------------------------------------------------

def _own_run(s):
    import activation_sparse_transformer_bf16_amd as tw

    c = s["case"]
    op = c["op"]
    if op == "quantize":
        return tw.twell_dequantize_mx4(tw.twell_quantize_mx4(s["x"]), s["x"].dtype)
    if op == "norm":
        n = tw.twell_rmsnorm_mx4(s["x"], s["weight"], eps=EPS, residual=s["residual"])
        out = {"y": n.y, "q": tw.twell_dequantize_mx4(n.q, s["x"].dtype)}
        if s["residual"] is not None:
            out["h"] = n.h
        return out
    if op == "product":
        return tw.twell_mx4_matmul(tw.Mx4Rows(*s["a"], c["K"]), tw.Mx4Rows(*s["b"], c["K"]), row_bias=s["bias"],
                                   dtype=TYPES[c["dtype"]])
    if "optimizer" not in s:
        s["optimizer"] = tw.TwellAdamW(s["weights"], s["m"], s["v"], s["m_scale"], s["v_scale"], s["master"],
                                       weight_decay=DECAY)
    opt = s["optimizer"]
    clip = tw.twell_grad_norm(s["grads"], MAX_NORM) if c["clip"] else None
    s["step"] += 1
    tw.twell_adamw_step(opt, s["grads"], lr=LR, step=s["step"], beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, clip=clip)
    m, v = (tw.twell_adamw_states(opt, torch.bfloat16) if c["bits"] == 8 else (opt.m, opt.v))
    out = [{"w": w, "m": a, "v": b} if x is None else {"w": w, "m": a, "v": b, "master": x}
           for w, a, b, x in zip(opt.weights, m, v, opt.master)]
    return out if clip is None else out + [clip]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "quantize":
        return _mx4_values(state["x"].float(), state["x"].dtype)
    if op == "norm":
        return _plain_norm(state)
    if op == "product":
        return _plain_product(state)
    return _plain_step(state)


def work(case):
    op = case["op"]
    s = 2 if case["dtype"] == "bf16" else 4
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * s, "flops": 4 * n}
    if op == "norm":
        n, d = case["T"] * case["d"], case["d"]
        # x, residual, h, y and the values returned for the 4 bits; the weight
        return {"bytes": n * s * (5 if case["residual"] else 3) + d * s, "flops": 8 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K / 2 + K / 32) + M * N * s + (4 * M if case["bias"] else 0), "flops": 2 * M * N * K}
    n = sum(_sizes(case))
    each = (2 if case["grad"] == "bf16" else 4) + (8 + s if case["master"] else 2 * s)
    # states read and written; 8-bit ones with a scale byte for each 32, and the values returned for them
    each += 16 if case["bits"] == 32 else 4 + 4 / 32 + 4
    return {"bytes": n * each, "flops": 20 * n}


# ---- 64 bits --------------------------------------------------------------------------

def _exact_mx4(z):
    """The nearest 4-bit values of rows z in 64 bits."""
    rows, cols = z.shape
    blocks = torch.cat((z, z.new_zeros(rows, -cols % 32)), 1).unflatten(1, (-1, 32))
    top = blocks.abs().max(dim=2, keepdim=True).values
    e = torch.ceil(torch.log2((top / 7).clamp_min(2.0 ** -126))).clamp(-126, 126)
    a = blocks.abs() * torch.exp2(-e)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=z.device)
    low = torch.bucketize(a, mids)  # a value between two levels goes to the lower one
    tie = (a == mids[low.clamp_max(6)]) & (low % 2 == 1) & (low < 7)
    level = torch.tensor(LEVELS, dtype=torch.float64, device=z.device)[low + tie]
    return (level * torch.sign(blocks) * torch.exp2(e)).flatten(1)[:, :cols]


def _exact_decode(rows, cols):
    q, scale = rows
    out = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
    for half in range(2):
        code = (q.long() >> (4 * half)) & 15
        field, part = (code & 7) >> 1, code & 1
        size = torch.where(field == 0, 0.5 * part, (1.0 + 0.5 * part) * torch.exp2(field.double() - 1.0))
        out[:, half::2] = torch.where(code >= 8, -size, size)
    e = torch.empty(q.shape[0], _ceil(cols, 32) // 32, dtype=torch.float64, device=q.device)
    for b in range(e.shape[1]):
        e[:, b] = scale[:, b // 16 * 16 + b % 4 * 4 + b // 4 % 4].double() - 127.0
    return out[:, :cols] * torch.exp2(e).repeat_interleave(32, dim=1)[:, :cols]


def _exact_state(x, dither, fields, positive):
    """Microscaled 8-bit values of x [n] in 64 bits: `fields` exponents, the topmost for the block's 2^E."""
    n = x.shape[0]
    a = torch.cat((x.abs(), x.new_zeros(-n % 32))).view(-1, 32)
    u = torch.cat(((dither.double() + 0.5) / 65536, x.new_zeros(-n % 32))).view(-1, 32)
    top = torch.ceil(torch.log2((a.max(dim=1, keepdim=True).values / 1.875).clamp_min(2.0 ** -87))).clamp(-87, 113)
    low = top - (fields - 2)
    e = torch.maximum(torch.floor(torch.log2(a.clamp_min(1e-300))), low)
    step = torch.exp2(e - 3)
    out = torch.floor(a / step + u) * step
    if positive:
        out = torch.where((a > 0) & (out == 0), torch.exp2(low - 3), out)
    return out.view(-1)[:n] * torch.sign(x)


def _exact_step(case, s):
    t = s["step"] + 1
    grads = [g.double() for g in s["grads"]]
    out = []
    factor = 1.0
    if case["clip"]:
        norm = math.sqrt(math.fsum(float((g * g).sum()) for g in grads))
        factor = min(1.0, MAX_NORM / norm)
    c1, c2 = -math.expm1(t * math.log(BETA1)), -math.expm1(t * math.log(BETA2))
    for i, g in enumerate(grads):
        g = g * factor
        m, v = s["m"][i].double(), s["v"][i].double()
        if case["bits"] == 8:
            def value(code, scale, fields):
                c = code.long() % (fields * 8)
                e = (c // 8).clamp_min(1) - 3
                part = c % 8 + 8 * (c >= 8)
                x = part.double() * torch.exp2((e - (fields - 1)).double())
                x = x * torch.exp2(scale.double() - 127).repeat_interleave(32)[:code.shape[0]]
                return torch.where(code.long() >= fields * 8, -x, x)
            m, v = value(s["m"][i], s["m_scale"][i], 16), value(s["v"][i], s["v_scale"][i], 32)
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g * g
        w = (s["master"][i] if case["master"] else s["weights"][i]).double()
        w = w - LR * DECAY * w - LR * (m / c1) / ((v / c2).sqrt() + ADAM_EPS)
        if case["bits"] == 8:
            bits = _random(t, i, g.shape[0])
            m, v = _exact_state(m, bits % 65536, 16, False), _exact_state(v, bits // 65536, 32, True)
        out.append({"w": w, "m": m, "v": v, "master": w} if case["master"] else {"w": w, "m": m, "v": v})
    if case["clip"]:
        out.append(torch.tensor([norm, factor], dtype=torch.float64))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_mx4(s["x"].double())
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        w = s["weight"].double()
        root = (h.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS).sqrt()
        # the definition rounds h w to 32 bits
        out = {"y": h / root * w, "q": _exact_mx4((h * w).float().double()) / root}
        if s["residual"] is not None:
            out["h"] = h
        return out
    if op == "step":
        return _exact_step(case, s)
    y = _exact_decode(s["a"], case["K"]).mm(_exact_decode(s["b"], case["K"]).t().contiguous())
    return y if s["bias"] is None else y + s["bias"].double()[:, None]
