"""Cases of a feed-forward block over 4-bit weights: the norm in front of it, its linear layers, and their gradients.

A weight [N, K] is held as packed E2M1 codes (K / 2 bytes a row, element 2k in the low nibble of byte k) with block
scales along K: NVFP4 (16-element blocks, E4M3 scale bytes, one fp32 tensor scale) or MXFP4 (32-element blocks, E8M0
scale bytes).  Activations are bf16, fp32, or MXFP8: E4M3 codes with one E8M0 scale for each 32 elements of a row.

Six kinds of case:
  linear       y = x W^T (+ bias)
  linear_back  dx = dy W
  gated        h = SiLU(x Wg^T) * (x Wu^T), Wg and Wu the two halves of one weight's rows
  gated_train  h, and from its gradient those of x and of the two products
  norm         s = x + residual, y = s / sqrt(mean(s^2) + eps) * w, as MXFP8 blocks or in x's type
  norm_train   y and s, and from their gradients those of x (and the residual: the same) and w
The stored sum s is rounded to x's type, and the norm is that of the stored sum.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = {"nvfp4": 16, "mxfp4": 32}
EPS = 1e-6


def _linear(name, op="linear", **kw):
    case = dict(name=name, op=op, format="nvfp4", rows=1, n=4096, k=4096, x="bf16", bias=False)
    case.update(kw)
    return case


def _norm(name, op="norm", **kw):
    case = dict(name=name, op=op, rows=1, d=8192, x="bf16", residual=True, mxfp8=False)
    case.update(kw)
    return case


def listed():
    return [
        # one user's token through a small layer: latency
        _linear("linear-token"),
        # the widest projection back to the hidden size, one token: a stream over the weight
        _linear("linear-down", format="mxfp4", n=8192, k=28672),
        # a serving batch's step, with a bias
        _linear("linear-batch", rows=24, n=8192, k=8192, bias=True),
        # drafted tokens of an fp32 model with odd sizes
        _linear("linear-odd", rows=7, n=1000, k=1360, x="f32"),
        # prompts of a batch, activations in 8 bits as the norm leaves them
        _linear("linear-prompt", format="mxfp4", rows=2048, n=8192, k=8192, x="mxfp8"),
        # the gradient that a frozen 4-bit layer hands on, adapters being trained beside it
        _linear("linear-back", op="linear_back", rows=1024, n=8192, k=8192),
        # one token through both wide projections of a large model
        _linear("gated-token", op="gated", n=28672, k=8192),
        # a serving batch, odd width
        _linear("gated-batch", op="gated", format="mxfp4", rows=40, n=10000, k=4096),
        # a training step of adapters around a frozen block: forward and backward
        _linear("gated-train", op="gated_train", rows=2048, n=8192, k=4096),
        # a serving batch's step, activations for 8-bit products
        _norm("norm-step", rows=64, mxfp8=True),
        # a batch of prompts
        _norm("norm-prompt", rows=8192, mxfp8=True),
        # a training step in fp32, odd sizes
        _norm("norm-train", op="norm_train", rows=4099, d=5000, x="f32"),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    op = rng.choice(("linear", "linear", "linear_back", "gated", "gated_train", "norm", "norm_train"))
    if op.startswith("norm"):
        eight = op == "norm" and rng.random() < 0.5
        d = 32 * log(2, 512) if eight else log(64, 16384)
        return dict(op=op, rows=min(log(1, 16384), 8192 * 8192 // d), d=d, x=rng.choice(("bf16", "f32")),
                    residual=rng.random() < 0.7, mxfp8=eight)
    fmt = rng.choice(("nvfp4", "mxfp4"))
    x = rng.choice(("bf16", "bf16", "f32") if op in ("linear_back", "gated_train") else ("bf16", "bf16", "f32", "mxfp8"))
    unit = 32 if x == "mxfp8" else BLOCK[fmt]
    gated = op.startswith("gated")
    n, k = log(128, 28672) // (2 if gated else 1), unit * log(256 // unit, 28672 // unit)
    if rng.random() < 0.5:
        n = max(64, n // 64 * 64)
    n = min(n, 235_000_000 // k)
    # products of the two training passes count twice; f32 activations cost several times as much
    most = 2.7e14 / ((2 if gated else 1) * (2 if op == "gated_train" else 1) * (4 if x == "f32" else 1) * 2 * n * k)
    return dict(op=op, format=fmt, rows=max(1, min(log(1, 4096), int(most))), n=n, k=k, x=x,
                bias=op == "linear" and rng.random() < 0.5)


def _size(kind):
    return {"bf16": 2.0, "f32": 4.0, "mxfp8": 1 + 1 / 32}[kind]


def work(case):
    op, m = case["op"], case["rows"]
    x = _size(case["x"])
    out = 4 if case["x"] == "f32" else 2
    if op == "norm":
        each = x * (1 + 2 * case["residual"]) + (_size("mxfp8") if case["mxfp8"] else out)
        return {"bytes": m * case["d"] * each + 4 * case["d"], "flops": m * case["d"] * 5}
    if op == "norm_train":
        # x, residual, the gradients of y and s in; y, s and the gradient of x out
        each = x * (1 + 2 * case["residual"] + 1 + case["residual"] + 2)
        return {"bytes": m * case["d"] * each + 8 * case["d"], "flops": m * case["d"] * 16}
    n, k = case["n"], case["k"]
    rows = 2 * n if op.startswith("gated") else n
    weight = rows * k * (0.5 + 1 / BLOCK[case["format"]])
    flops = 2 * m * rows * k
    if op == "gated_train":
        # x and the gradient of h in; h, the gradients of x and of the products out
        return {"bytes": weight + m * x * (2 * k + 4 * n), "flops": 2 * flops}
    if op == "linear_back":
        return {"bytes": weight + m * x * (n + k), "flops": flops}
    return {"bytes": weight + m * (x * k + out * n) + out * n * case["bias"], "flops": flops}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    m, op = case["rows"], case["op"]
    state = {"case": case}
    if op.startswith("norm"):
        d, t = case["d"], DTYPES[case["x"]]
        # a few channels far larger than the others, as residual streams have them
        big = 1 + 20 * (torch.rand(d, generator=gen, device=dev) > 0.995)
        state["x"] = normal(m, d).to(t)
        state["residual"] = (normal(m, d) * big).to(t) if case["residual"] else None
        state["w"] = (1 + 0.2 * normal(d)).to(t)
        if op == "norm_train":
            state["dy"] = (0.01 * normal(m, d)).to(t)
            state["ds"] = (0.01 * normal(m, d)).to(t) if case["residual"] else None
        return state
    fmt, k = case["format"], case["k"]
    n = 2 * case["n"] if op.startswith("gated") else case["n"]
    # The codes of a Gaussian block scaled to its largest value are close to uniform over the sixteen of them, and
    # their scales spread over about two octaves; the tensor scale brings products of unit activations to about one.
    codes = torch.randint(0, 256, (n, k // 2), generator=gen, device=dev, dtype=torch.uint8)
    low = 0x38 if fmt == "nvfp4" else 127 - 2 - int(math.log2(k)) // 2
    scales = torch.randint(low, low + (17 if fmt == "nvfp4" else 3), (n, k // BLOCK[fmt]), generator=gen, device=dev,
                           dtype=torch.uint8)
    tensor_scale = torch.full((1,), 0.13 / math.sqrt(k), device=dev) if fmt == "nvfp4" else None
    state["weight"] = (fmt, codes, scales, tensor_scale)
    if own:     # the handle that a program makes when it loads the weight
        import fp4_block_scaled_row_amd as fq
        state["handle"] = fq.Fp4Weight(*state["weight"])
    if op == "linear_back":
        state["dy"] = (0.01 * normal(m, n)).to(DTYPES[case["x"]])
        return state
    x = normal(m, k) * (1 + 7 * (torch.rand(k, generator=gen, device=dev) > 0.99))
    if case["x"] == "mxfp8":
        state["x"] = _quantised(x)
    else:
        state["x"] = x.to(DTYPES[case["x"]])
    state["bias"] = normal(n).to(_out(case)) if case["bias"] else None
    if op == "gated_train":
        state["dh"] = (0.01 * normal(m, case["n"])).to(DTYPES[case["x"]])
    return state


def _out(case):
    return torch.float32 if case["x"] == "f32" else torch.bfloat16


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(state, case, op)
    if op.startswith("norm"):
        return _plain_norm(state, case)
    w = _weight(*state["weight"])
    t = _out(case)
    if op == "linear_back":
        return torch.mm(state["dy"].float(), w).to(t)
    x = _values(*state["x"]) if case["x"] == "mxfp8" else state["x"].float()
    y = torch.mm(x, w.t())
    if op == "linear":
        return (y if state["bias"] is None else y + state["bias"].float()).to(t)
    gate, up = y[:, :case["n"]], y[:, case["n"]:]
    sig = 1 / (1 + torch.exp(-gate))
    h = (gate * sig * up).to(t)
    if op == "gated":
        return h
    dh = state["dh"].float()
    dy = torch.cat((dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig), 1)
    return h, torch.mm(dy, w).to(t), dy.to(t)


def _run_own(state, case, op):
    import fp4_block_scaled_row_amd as fq
    if op == "norm":
        r = fq.rms_norm(state["x"], state["w"], residual=state["residual"], eps=EPS,
                        quantize="mxfp8" if case["mxfp8"] else None)
        y = fq.dequantize("mxfp8", *r.out, out_dtype=_out(case)) if case["mxfp8"] else r.out
        return (y, r.summed) if case["residual"] else y
    if op == "norm_train":
        r = fq.rms_norm(state["x"], state["w"], residual=state["residual"], eps=EPS, return_rstd=True)
        s = r.summed if case["residual"] else state["x"]
        dx, dw = fq.rms_norm_backward(state["dy"], s, state["w"], r.rstd, dsummed=state["ds"])
        return (r.out, s, dx, dw) if case["residual"] else (r.out, dx, dw)
    w = state["handle"]
    if op == "linear_back":
        return fq.fp4_linear_backward(state["dy"], w)
    x = fq.Mx8Result(*state["x"]) if case["x"] == "mxfp8" else state["x"]
    if op == "linear":
        return fq.fp4_linear(x, w, bias=state["bias"])
    if op == "gated":
        return fq.fp4_gated(x, w)
    h, products = fq.fp4_gated(x, w, return_products=True)
    dx, dproducts = fq.fp4_gated_backward(state["dh"], products, w)
    return h, dx, dproducts


# ---------------------------------------------------------------------------------------------- the plain form

def _scale_of(fmt, byte):
    if fmt == "nvfp4":
        return byte.view(torch.float8_e4m3fn).float()
    return torch.ldexp(torch.ones((), device=byte.device), byte.int() - 127)


def _weight(fmt, codes, scales, tensor_scale):
    lattice = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    both = torch.cat((lattice, -lattice))
    pair = torch.stack((both[None].expand(16, 16), both[:, None].expand(16, 16)), -1).reshape(256, 2)
    s = _scale_of(fmt, scales)
    if fmt == "nvfp4":
        s = s * tensor_scale
    x = pair[codes.int()].reshape(*scales.shape, BLOCK[fmt])
    return x.mul_(s[..., None]).reshape(scales.shape[0], -1)


def _quantised(y):
    """MXFP8 of fp32 rows: E4M3 codes as bytes, and E8M0 scales 2^(floor(log2 of the block's largest) - 8)."""
    b = y.unflatten(1, (-1, 32))
    most = b.abs().amax(-1)
    e = torch.where(most > 0, (most.view(torch.int32) >> 23) - 127 - 8, 0).clamp(min=-127)
    q = torch.ldexp(b, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(y.shape), (e + 127).to(torch.uint8)


def _values(codes, scales):
    q = codes.view(torch.float8_e4m3fn).float().unflatten(1, (-1, 32))
    return torch.ldexp(q, scales.int()[..., None] - 127).reshape(codes.shape)


def _plain_norm(state, case):
    t = _out(case)
    s = state["x"].float()
    if case["residual"]:
        s = (s + state["residual"].float()).to(t).float()
    w = state["w"].float()
    rstd = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + EPS)
    hat = s * rstd
    y = hat * w
    if case["op"] == "norm":
        y = _values(*_quantised(y)).to(t) if case["mxfp8"] else y.to(t)
        return (y, s.to(t)) if case["residual"] else y
    dy = state["dy"].float()
    g = dy * w
    dx = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
    if case["residual"]:
        dx = dx + state["ds"].float()
    dw = (dy * hat).sum(0).to(t)
    return (y.to(t), s.to(t), dx.to(t), dw) if case["residual"] else (y.to(t), dx.to(t), dw)


# ---------------------------------------------------------------------------------------------- in 64 bits

def _exact_scale(fmt, byte):
    b = byte.long()
    if fmt == "mxfp4":
        return torch.exp2(b.double() - 127)
    e, m = b >> 3, (b & 7).double()
    return torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e.double() - 7) * (1 + m / 8))


def _exact_weight(fmt, codes, scales, tensor_scale):
    """Element by element from the bits: sign, two exponent bits of bias 1, one mantissa bit."""
    rows = []
    for c, s in zip(codes.split(4096), scales.split(4096)):
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2).int()
        e, m = (c >> 1) & 3, (c & 1).double()
        x = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m)) * (1 - 2 * (c >> 3))
        x = x * _exact_scale(fmt, s).repeat_interleave(BLOCK[fmt], -1)
        rows.append(x * tensor_scale.double() if fmt == "nvfp4" else x)
    return torch.cat(rows)


def _exact_e4m3(codes):
    c = codes.int()
    e, m = (c >> 3) & 15, (c & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e.double() - 7) * (1 + m / 8))
    return x * (1 - 2 * (c >> 7))


def _exact_mxfp8(y):
    """The values that MXFP8 blocks of y stand for: the nearest E4M3 number times the block's power of two."""
    b = y.unflatten(1, (-1, 32))
    most = b.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(torch.where(most > 0, most, 256.0))        # most = m 2^e, m in [0.5, 1)
    scale = torch.exp2((e.double() - 1 - 8).clamp(min=-127))
    q = b / scale
    _, e = torch.frexp(q)
    step = torch.exp2((e.double() - 1).clamp(min=-6) - 3)
    return ((torch.round(q / step) * step).clamp(-448, 448) * scale).flatten(1)


def exact(case, seed):
    if work(case)["flops"] > 6e14:
        return None
    state = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(state, case)
    w = _exact_weight(*state["weight"])
    if op == "linear_back":
        return state["dy"].double() @ w
    if case["x"] == "mxfp8":
        codes, scales = state["x"]
        x = _exact_e4m3(codes) * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
    else:
        x = state["x"].double()
    if op == "linear":
        y = x @ w.T
        return y if state["bias"] is None else y + state["bias"].double()
    gate, up = x @ w[:case["n"]].T, x @ w[case["n"]:].T
    h = gate * torch.sigmoid(gate) * up
    if op == "gated":
        return h
    # derivatives of SiLU(gate) * up
    sig, dh = torch.sigmoid(gate), state["dh"].double()
    d_gate = dh * up * (sig + gate * sig * torch.sigmoid(-gate))
    d_up = dh * gate * sig
    return h, d_gate @ w[:case["n"]] + d_up @ w[case["n"]:], torch.cat((d_gate, d_up), 1)


def _exact_norm(state, case):
    s = state["x"].double()
    if case["residual"]:
        s = (state["x"].double() + state["residual"].double()).to(_out(case)).double()
    w, d = state["w"].double(), case["d"]
    r = torch.rsqrt(s.square().sum(1) / d + EPS)
    y = s * r[:, None] * w
    if case["op"] == "norm":
        y = _exact_mxfp8(y) if case["mxfp8"] else y
        return (y, s) if case["residual"] else y
    # y_i = s_i r w_i with dr/ds_j = -r^3 s_j / d
    dy = state["dy"].double()
    along = (dy * w * s).sum(1) * r ** 3 / d
    dx = dy * w * r[:, None] - s * along[:, None]
    if case["residual"]:
        dx = dx + state["ds"].double()
    dw = (dy * s * r[:, None]).sum(0)
    return (y, s, dx, dw) if case["residual"] else (y, dx, dw)
