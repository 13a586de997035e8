"""Cases of the 4-bit key/value cache: storing tokens into it, reading them back, and attention over it.

A cache holds keys and values in pages.  Page p, head h, token offset o of a plane is a row of packed E2M1 codes
(head_dim / 2 bytes, element 2k in the low nibble of byte k) or of block scales: NVFP4 (16-element blocks, E4M3 scale
bytes, one fp32 tensor scale each for keys and values) or MXFP4 (32-element blocks, E8M0 scale bytes).  Sequence b's
token t lies in page page_table[b][t // page] at offset t % page.

Three kinds of case:
  store   quantise new tokens into their slots (keys rotated by the normalised 128-point Hadamard transform where the
          case says so) and read the same tokens back as values, in the keys' original basis
  read    the values of whole sequences, gathered into dense rows
  attend  softmax(scale q k^T) v over the cache, heads in groups, causal from the sequence's end, optionally only the
          last `window` tokens; a row that sees no token is zero and its log-sum-exp minus infinity
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def _attend(name, **kw):
    case = dict(name=name, op="attend", format="nvfp4", head_dim=128, q_heads=32, kv_heads=8, seqs=1, longest=1024,
                queries=1, page=64, dtype="bf16", rotate=False, window=0, idle=False, lse=False)
    case.update(kw)
    return case


def _rows(name, op, **kw):
    case = dict(name=name, op=op, format="nvfp4", head_dim=128, kv_heads=8, seqs=1, longest=1024, page=64,
                dtype="bf16", rotate=False)
    case.update(kw)
    return case


def listed():
    return [
        # one new token for each of 64 running sequences: a decode step's append, all latency
        _rows("store-step", "store", seqs=64, longest=1, page=16, rotate=True),
        # four prompts' chunks appended at once
        _rows("store-chunk", "store", seqs=4, longest=2048, rotate=True),
        # one odd-length prompt in fp32, head_dim 96, pages that are no power of two
        _rows("store-odd", "store", format="mxfp4", head_dim=96, kv_heads=5, longest=1999, page=24, dtype="f32"),
        # a prefix read back for a layer that wants dense fp32 keys and values
        _rows("read-prefix", "read", format="mxfp4", head_dim=64, longest=4093, page=32, dtype="f32"),
        # a batch of long contexts read back as bf16
        _rows("read-batch", "read", seqs=16, longest=16384, rotate=True),
        # one user, short context: latency
        _attend("decode-one", longest=1023, page=16, rotate=True),
        # a serving batch, ragged, with an idle slot
        _attend("decode-batch", seqs=64, longest=8192, rotate=True, idle=True),
        # two very long contexts
        _attend("decode-long", format="mxfp4", q_heads=64, seqs=2, longest=131071, page=128),
        # four draft tokens verified per sequence, one shared key/value head, sliding window
        _attend("decode-draft", format="mxfp4", head_dim=256, q_heads=16, kv_heads=1, seqs=16, longest=6000, queries=4,
                page=24, window=4095),
        # fp32 model without shared heads, log-sum-exp kept for joining with other parts of the context
        _attend("decode-f32", head_dim=64, q_heads=12, kv_heads=12, seqs=8, longest=2000, page=40, dtype="f32",
                lse=True),
        # a whole prompt
        _attend("prefill", longest=4096, queries=4096, rotate=True),
        # chunks of several prompts over what is cached of them, group of five heads
        _attend("extend", format="mxfp4", q_heads=40, seqs=4, longest=16000, queries=1000),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    fmt, dim = rng.choice(("nvfp4", "mxfp4")), rng.choice((64, 96, 128, 128, 256))
    base = dict(format=fmt, head_dim=dim, page=rng.choice((16, 24, 32, 40, 64, 128)),
                dtype=rng.choice(("bf16", "bf16", "f32")), rotate=dim % 128 == 0 and rng.random() < 0.5)
    op = rng.choice(("store", "read", "attend", "attend", "attend"))
    heads = rng.choice((1, 2, 5, 8, 12))
    if op != "attend":
        seqs = log(1, 64)
        longest = log(1, 4096)
        return dict(base, op=op, kv_heads=heads, seqs=seqs, longest=min(longest, 131072 // seqs))
    group = rng.choice((1, 4, 5, 8, 16))
    seqs, queries = log(1, 64), 1
    if rng.random() < 0.3:
        queries = rng.randint(2, 8)
    elif rng.random() < 0.5:
        queries = log(9, 2048)
        seqs = min(seqs, 8)
    longest = max(queries, log(16, 131071))
    # (sequence, token) pairs and score pairs stay below those of the largest listed cases
    longest = max(queries, min(longest, 262144 // seqs, 1 << 18, int(5e8 / (queries * seqs * heads * group))))
    return dict(base, op=op, q_heads=heads * group, kv_heads=heads, seqs=seqs, longest=longest, queries=queries,
                window=rng.choice((0, 0, 0, log(1, 8192))), idle=seqs > 2 and rng.random() < 0.3,
                lse=rng.random() < 0.3)


def _lengths(case):
    """Tokens in the cache and new queries of every sequence: a property of the case, not of the seed."""
    rng = random.Random(case["seqs"] * 1000003 + case["longest"])
    lens = [case["longest"]] + [max(1, int(case["longest"] * rng.uniform(0.25, 1.0))) for _ in range(case["seqs"] - 1)]
    if case["op"] != "attend":
        return lens, lens
    most = case["queries"]
    new = [most] + [rng.randint((most + 1) // 2, most) for _ in range(case["seqs"] - 1)]
    lens = [max(n, m) for n, m in zip(lens, new)]
    if case["idle"]:
        lens[-1] = 0
    return lens, new


def _visible(case, n, m):
    """Tokens of a sequence of n that its m queries see: those seen by any, and (query, token) pairs."""
    w = case["window"] or 1 << 60
    seen = [max(0, min(n - m + i + 1, w)) for i in range(m)]
    first = max(0, n - m + 1 - w)
    return max(0, n - first), sum(seen)


def work(case):
    dim, heads, esz = case["head_dim"], case["kv_heads"], 2 if case["dtype"] == "bf16" else 4
    row = dim // 2 + dim // BLOCK[case["format"]]
    lens, new = _lengths(case)
    if case["op"] != "attend":
        values = 2 * sum(lens) * heads * dim
        held = 2 * sum(lens) * heads * row
        if case["op"] == "read":
            return {"bytes": held + values * esz, "flops": values * (2 + 3.5 * case["rotate"])}
        # store: values in, the cache written, read again and values out
        return {"bytes": 2 * held + 2 * values * esz, "flops": values * (4 + 7 * case["rotate"])}
    counts = [_visible(case, n, m) for n, m in zip(lens, new)]
    rows = sum(new) * case["q_heads"]
    return {"bytes": 2 * heads * row * sum(t for t, _ in counts) + 2 * rows * dim * esz + 4 * rows * case["lse"],
            "flops": 4 * dim * case["q_heads"] * sum(p for _, p in counts)}


def _cumulative(counts, device):
    return torch.tensor([0] + counts, device=device).cumsum(0).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dim, heads, page, dtype = case["head_dim"], case["kv_heads"], case["page"], DTYPES[case["dtype"]]
    block = BLOCK[case["format"]]
    lens, new = _lengths(case)
    per = max(1, -(-max(lens) // page))
    pages = case["seqs"] * per + 3
    table = torch.randperm(pages, generator=gen, device=dev)[: case["seqs"] * per].to(torch.int32).view(case["seqs"], per)

    def bytes_(lo, hi, width):
        return torch.randint(lo, hi, (pages, heads, page, width), generator=gen, device=dev, dtype=torch.uint8)

    # The codes of a Gaussian block scaled to its largest value are close to uniform over the sixteen of them.  Scales
    # spread over two octaves, as those of keys with strong and weak channels do.  The tensor scales are powers of two
    # (a calibration rounds them up) that bring the values to about one.
    span = (0x30, 0x41) if case["format"] == "nvfp4" else (123, 127)
    if case["op"] == "store":
        lo = torch.zeros
        k_codes, k_scales, v_codes, v_scales = (lo((pages, heads, page, w), device=dev, dtype=torch.uint8)
                                                for w in (dim // 2, dim // block, dim // 2, dim // block))
    else:
        k_codes, v_codes = bytes_(0, 256, dim // 2), bytes_(0, 256, dim // 2)
        k_scales, v_scales = bytes_(*span, dim // block), bytes_(*span, dim // block)
    one = 0.25 if case["op"] != "store" else 2.0 ** -8
    state = {"case": case, "table": table, "page": page, "lens_host": lens, "new_host": new,
             "lens": torch.tensor(lens, device=dev, dtype=torch.int32),
             "cache": (case["format"], k_codes, k_scales, v_codes, v_scales,
                       torch.full((1,), one, device=dev), torch.full((1,), one / 2, device=dev)),
             "total": sum(new), "cu": _cumulative(new, dev)}
    if own:     # the handle over the planes that a serving program makes when it allocates them
        import fp4_block_scaled_row_amd as fq
        state["handle"] = fq.KvCache(*state["cache"])
    # padded positions, for the plain form: row (b, i) of the packed rows, and whether it is there
    widest = max(new)
    at = torch.arange(widest, device=dev)
    state["there"] = at[None] < torch.tensor(new, device=dev)[:, None]
    if case["op"] == "attend":
        state["q"] = 1.5 * torch.randn((sum(new), case["q_heads"], dim), generator=gen, device=dev)
        state["q"] = state["q"].to(dtype)
        state["tokens"] = torch.arange(max(1, max(lens)), device=dev)
        state["scale"] = dim ** -0.5
        return state
    rows = torch.arange(case["seqs"], device=dev)[:, None].expand(-1, widest)[state["there"]]
    pos = at[None].expand(case["seqs"], -1)[state["there"]]
    state["slots"] = table[rows, pos // page].long() * page + pos % page
    if case["op"] == "store":
        # keys and values as a projection leaves them: one matrix [tokens, 2, heads, dim], a few channels far larger
        kv = torch.randn((sum(lens), 2, heads, dim), generator=gen, device=dev)
        kv[:, 0] *= 1 + 7 * (torch.rand((heads, dim), generator=gen, device=dev) > 0.97)
        kv = kv.to(dtype)
        state["k"], state["v"] = kv[:, 0], kv[:, 1]
    return state


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "store":
        return _plain_store(state, case)
    if case["op"] == "read":
        return _plain_read(state, case)
    return _plain_attend(state, case)


def _run_own(state, case):
    import fp4_block_scaled_row_amd as fq
    cache = state["handle"]
    rotation = "fwht128" if case["rotate"] else None
    if case["op"] == "attend":
        return fq.kv_cache_attention(state["q"], cache, state["table"], state["lens"],
                                     cu_q=None if case["queries"] == 1 else state["cu"], max_q=case["queries"],
                                     scale=state["scale"], causal=True, window=case["window"], rotation=rotation,
                                     return_lse=case["lse"])
    if case["op"] == "store":
        fq.kv_cache_write(cache, state["k"], state["v"], state["slots"], rotation=rotation)
    return fq.kv_cache_read(cache, state["table"], state["cu"], total=state["total"], rotation=rotation,
                            out_dtype=DTYPES[case["dtype"]])


# ---------------------------------------------------------------------------------------------- the plain form

def _butterfly(x, h):
    """One stage of the Hadamard transform: elements h apart become their sum and difference."""
    y = x.reshape(*x.shape[:-1], -1, 2, h)
    a, b = y[..., 0, :], y[..., 1, :]
    return torch.stack((a + b, a - b), -2).reshape(x.shape)


def _rotated(x, rotate):
    """Normalised Hadamard transform of each 128 elements, stages from neighbours outwards, scaled once."""
    if not rotate:
        return x
    y = _butterfly(_butterfly(_butterfly(_butterfly(x, 1), 2), 4), 8)
    return _butterfly(_butterfly(_butterfly(y, 16), 32), 64) * (1 / math.sqrt(128))


def _scale_of(fmt, byte):
    if fmt == "nvfp4":
        return byte.view(torch.float8_e4m3fn).float()
    return torch.ldexp(torch.ones((), device=byte.device), byte.int() - 127)


def _values(fmt, codes, scales, tensor_scale):
    lattice = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    both = torch.cat((lattice, -lattice))
    pair = torch.stack((both[None].expand(16, 16), both[:, None].expand(16, 16)), -1).reshape(256, 2)
    x = pair[codes.long()].reshape(*scales.shape, BLOCK[fmt]) * _scale_of(fmt, scales)[..., None]
    x = x.reshape(*scales.shape[:-1], -1)
    return x * tensor_scale if fmt == "nvfp4" else x


def _quantised(fmt, x, tensor_scale):
    """(codes, scale bytes) of fp32 x; the quotients' roundings decide every tie exactly where the tensor scale is a
    power of two: a neighbour of a tie is over half a unit in the last place from it after the division."""
    x = x.reshape(*x.shape[:-1], -1, BLOCK[fmt])
    most = x.abs().amax(-1)
    if fmt == "nvfp4":
        byte = (most / (6 * tensor_scale)).clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        step = _scale_of(fmt, byte) * tensor_scale
    else:
        power = (most.view(torch.int32) >> 23) - 127                       # floor(log2), of normal values
        byte = torch.where(most > 0, (power - 2).clamp(min=-127), 0).add(127).to(torch.uint8)
        step = _scale_of(fmt, byte)
    a = torch.where(step[..., None] > 0, x.abs() / step[..., None], 0.0)
    mag = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    code = (mag + 8 * torch.signbit(x)).to(torch.uint8).reshape(*x.shape[:-2], -1)
    return code[..., ::2] | code[..., 1::2] << 4, byte


def _plain_read(state, case):
    fmt, kc, ks, vc, vs, kg, vg = state["cache"]
    page, offset = state["slots"] // state["page"], state["slots"] % state["page"]
    k = _rotated(_values(fmt, kc[page, :, offset], ks[page, :, offset], kg), case["rotate"])
    v = _values(fmt, vc[page, :, offset], vs[page, :, offset], vg)
    return k.to(DTYPES[case["dtype"]]), v.to(DTYPES[case["dtype"]])


def _plain_store(state, case):
    fmt, kc, ks, vc, vs, kg, vg = state["cache"]
    page, offset = state["slots"] // state["page"], state["slots"] % state["page"]
    kc[page, :, offset], ks[page, :, offset] = _quantised(fmt, _rotated(state["k"].float(), case["rotate"]), kg)
    vc[page, :, offset], vs[page, :, offset] = _quantised(fmt, state["v"].float(), vg)
    return _plain_read(state, case)


def _plain_attend(state, case):
    fmt, kc, ks, vc, vs, kg, vg = state["cache"]
    seqs, heads, dim, group = case["seqs"], case["kv_heads"], case["head_dim"], case["q_heads"] // case["kv_heads"]
    t = state["tokens"]
    page, offset = state["table"].long()[:, t // state["page"]], (t % state["page"])[None]
    k = _values(fmt, kc[page, :, offset], ks[page, :, offset], kg)      # [seqs, tokens, heads, dim]
    v = _values(fmt, vc[page, :, offset], vs[page, :, offset], vg)
    there = state["there"]
    q = torch.zeros((seqs, there.shape[1], heads, group, dim), device=k.device)
    q[there] = _rotated(state["q"].float(), case["rotate"]).reshape(-1, heads, group, dim)
    q = q.permute(0, 2, 1, 3, 4).reshape(seqs * heads, -1, dim)
    k = k.permute(0, 2, 3, 1).reshape(seqs * heads, dim, -1)
    v = v.permute(0, 2, 1, 3).reshape(seqs * heads, -1, dim)
    s = (torch.bmm(q, k) * state["scale"]).view(seqs, heads, -1, group, t.numel())
    last = (state["lens"] - (state["cu"][1:] - state["cu"][:-1]))[:, None] + torch.arange(there.shape[1], device=k.device)
    sees = t <= last[..., None]                                            # [seqs, queries, tokens]
    if case["window"]:
        sees = sees & (t > last[..., None] - case["window"])
    s = torch.where(sees[:, None, :, None], s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(seqs * heads, -1, t.numel()), v).view(seqs, heads, -1, group, dim)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 2, 1, 3, 4)[there].reshape(-1, heads * group, dim).to(DTYPES[case["dtype"]])
    if not case["lse"]:
        return o
    lse = (torch.log(total) + top)[..., 0]
    return o, lse.permute(0, 2, 1, 3)[there].reshape(-1, heads * group)


# ---------------------------------------------------------------------------------------------- in 64 bits

def _exact_element(code):
    """E2M1 from its bits: sign, two exponent bits of bias 1, one mantissa bit."""
    e, m, sign = (code >> 1) & 3, code & 1, 1 - 2 * (code >> 3).double()
    return sign * torch.where(e == 0, 0.5 * m.double(), torch.exp2(e.double() - 1) * (1 + 0.5 * m.double()))


def _exact_scale(fmt, byte):
    b = byte.long()
    if fmt == "mxfp4":
        return torch.exp2(b.double() - 127)
    e, m = b >> 3, (b & 7).double()
    return torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e.double() - 7) * (1 + m / 8))


def _exact_rows(fmt, codes, scales, tensor_scale):
    c = codes.long()
    x = _exact_element(torch.stack((c & 15, c >> 4), -1).flatten(-2))
    x = x * _exact_scale(fmt, scales).repeat_interleave(BLOCK[fmt], -1)
    return x * tensor_scale.double() if fmt == "nvfp4" else x


def _exact_rotated(x, rotate):
    if not rotate:
        return x
    i = torch.arange(128, device=x.device)
    common = i[:, None] & i[None]
    parity = sum((common >> b) & 1 for b in range(7)) % 2
    h = (1 - 2 * parity).double() / math.sqrt(128)
    return (x.unflatten(-1, (-1, 128)) @ h).flatten(-2)


def _exact_stored(fmt, x, tensor_scale):
    """What the cache stands for after x was quantised into it."""
    b = x.unflatten(-1, (-1, BLOCK[fmt]))
    most = b.abs().amax(-1)
    g = tensor_scale.double()
    if fmt == "nvfp4":
        grid = _exact_scale(fmt, torch.arange(127, device=x.device))
        scale = grid[_nearest_even(most / (6 * g), grid)] * g
    else:
        e = torch.floor(torch.log2(torch.where(most > 0, most, 4.0))) - 2
        e = e + ((torch.exp2(e + 3) <= most) & (most > 0)).double() - ((torch.exp2(e + 2) > most) & (most > 0)).double()
        scale = torch.exp2(e.clamp(min=-127))
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device, dtype=torch.float64)
    a = torch.where(scale[..., None] > 0, b.abs() / scale[..., None], 0.0)
    return (grid[_nearest_even(a, grid)] * scale[..., None] * torch.sign(b)).flatten(-2)


def _nearest_even(a, grid):
    """Index of the grid point nearest to a; a tie goes to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.searchsorted(mid, a.contiguous()), torch.searchsorted(mid, a.contiguous(), right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def exact(case, seed):
    state = prepare(case, seed)
    fmt, kc, ks, vc, vs, kg, vg = state["cache"]
    if case["op"] == "store":
        k = _exact_stored(fmt, _exact_rotated(state["k"].double(), case["rotate"]), kg)
        return _exact_rotated(k, case["rotate"]), _exact_stored(fmt, state["v"].double(), vg)
    if case["op"] == "read":
        page, offset = state["slots"] // state["page"], state["slots"] % state["page"]
        k = _exact_rows(fmt, kc[page, :, offset], ks[page, :, offset], kg)
        return _exact_rotated(k, case["rotate"]), _exact_rows(fmt, vc[page, :, offset], vs[page, :, offset], vg)
    heads, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    q = _exact_rotated(state["q"].double(), case["rotate"])
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, device=q.device, dtype=torch.float64)
    begin = 0
    for b, (n, m) in enumerate(zip(state["lens_host"], state["new_host"])):
        t = torch.arange(n, device=q.device)
        page, offset = state["table"][b].long()[t // state["page"]], t % state["page"]
        last = n - m + torch.arange(m, device=q.device)
        sees = t[None] <= last[:, None]
        if case["window"]:
            sees &= t[None] > last[:, None] - case["window"]
        for h in range(heads if n else 0):
            k = _exact_rows(fmt, kc[page, h, offset], ks[page, h, offset], kg)
            v = _exact_rows(fmt, vc[page, h, offset], vs[page, h, offset], vg)
            mine = slice(h * group, (h + 1) * group)
            s = q[begin:begin + m, mine].flatten(0, 1) @ k.T * state["scale"]
            s = s.masked_fill(~sees.repeat_interleave(group, 0), -math.inf)
            z = torch.logsumexp(s, -1, keepdim=True)
            o = torch.exp(s - z.clamp(min=-1e300)) @ v
            out[begin:begin + m, mine], lse[begin:begin + m, mine] = o.view(m, group, -1), z.view(m, group)
        begin += m
    return (out, lse) if case["lse"] else out
