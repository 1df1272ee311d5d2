"""Measured cases of the layer's microscaled (MX) operators: quantisation to 4 and 8 bits and back, the residual's
addition with the root-mean-square norm and its 8-bit output, and the experts' products on microscaled operands.

An MX block is 32 consecutive elements of a row with one power-of-two scale; its elements are held as e2m1 (4 bits,
"fp4") or e4m3 (8 bits, "fp8").  ``run`` computes an operator from elementary torch operations in 32 bits, or, where
``own`` is set, calls the package's kernels.
"""
import math

import torch

own = False

BLOCK = 32
EMAX = {"fp4": 2, "fp8": 8}     # largest exponent of the element types
TOP = {"fp4": 6.0, "fp8": 448.0}
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One decode batch's hidden states to 8 bits: latency.
        {"name": "quantise decode batch", "op": "quantise", "dtype": "bf16", "format": "fp8", "rows": 8, "cols": 3584},
        # fp32 activations of an odd number of tokens at the capacity layer's inner size, to 4 bits.
        {"name": "quantise f32 odd", "op": "quantise", "dtype": "f32", "format": "fp4", "rows": 4099, "cols": 1408},
        # All of one projection's expert weights (32 x 5632 rows), once at load: the largest.
        {"name": "quantise weights", "op": "quantise", "dtype": "bf16", "format": "fp4", "rows": 32 * 5632, "cols": 2048},
        # The norm before the decode layer: 8 tokens.
        {"name": "norm decode", "op": "norm", "dtype": "bf16", "format": "fp8", "tokens": 8, "hidden": 3584, "residual": True},
        # A first layer's norm (no residual yet) in fp32, odd token count.
        {"name": "norm f32 odd", "op": "norm", "dtype": "f32", "format": "fp8", "tokens": 2049, "hidden": 2048, "residual": False},
        # The norm before a long prefill.
        {"name": "norm prefill", "op": "norm", "dtype": "bf16", "format": "fp8", "tokens": 16384, "hidden": 4096, "residual": True},
        # One token through its two experts: the smallest products.
        {"name": "experts token fp8", "op": "experts", "dtype": "bf16", "format": "fp8", "tokens": 1, "hidden": 3584,
         "inner": 2560, "experts": 64, "topk": 2},
        # The decode batch: a weight stream over most of 16 experts.
        {"name": "experts decode fp4", "op": "experts", "dtype": "bf16", "format": "fp4", "tokens": 8, "hidden": 3584,
         "inner": 2560, "experts": 64, "topk": 2},
        # A ragged middle: a few dozen rows for each expert.
        {"name": "experts ragged fp8", "op": "experts", "dtype": "bf16", "format": "fp8", "tokens": 333, "hidden": 2048,
         "inner": 1408, "experts": 32, "topk": 4},
        # The prefill layer with 8-bit activations.
        {"name": "experts prefill fp8", "op": "experts", "dtype": "bf16", "format": "fp8", "tokens": 8192, "hidden": 2048,
         "inner": 5632, "experts": 32, "topk": 2},
        # The largest layer with 4-bit activations.
        {"name": "experts large fp4", "op": "experts", "dtype": "bf16", "format": "fp4", "tokens": 16384, "hidden": 4096,
         "inner": 14336, "experts": 64, "topk": 2},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantise", "norm", "experts", "experts"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    form = rng.choice(["fp4", "fp8"])
    if op == "quantise":
        return {"op": op, "dtype": dtype, "format": form, "rows": _spread(rng, 1, 40000), "cols": 32 * _spread(rng, 2, 256)}
    if op == "norm":
        return {"op": op, "dtype": dtype, "format": rng.choice(["fp8", "fp8", "fp4"]), "tokens": _spread(rng, 1, 14000),
                "hidden": 64 * _spread(rng, 1, 64), "residual": rng.random() < 0.75}
    experts = rng.choice([1, 5, 8, 16, 32, 64])
    return {"op": op, "dtype": "bf16", "format": form, "tokens": _spread(rng, 1, 12000), "hidden": 64 * _spread(rng, 4, 64),
            "inner": 64 * _spread(rng, 4, 100), "experts": experts, "topk": min(experts, rng.choice([1, 2, 2, 4]))}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _encode(values, form):
    """Code bytes of values that the element type holds exactly (two e2m1 to a byte, the even element low)."""
    if form == "fp8":
        return values.to(torch.float8_e4m3fn).view(torch.uint8)
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=values.device)
    code = torch.bucketize(values.abs(), grid, out_int32=True).to(torch.uint8) | (torch.signbit(values).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _random_mx(g, shape, scale, form):
    """Codes and scale bytes of normal values, as the quantisation gives them; chunked, so that large weights fit."""
    rows, cols = math.prod(shape[:-1]), shape[-1]
    codes = torch.empty((rows, cols // 2 if form == "fp4" else cols), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, cols // BLOCK), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // cols)
    for at in range(0, rows, step):
        n = min(step, rows - at)
        q, e = _quantise(torch.randn((n, cols), generator=g, device="cuda") * scale, form)
        codes[at:at + n] = _encode(q, form).view(n, -1)
        scales[at:at + n] = (e + 127).to(torch.uint8)
    return codes.view(*shape[:-1], -1), scales.view(*shape[:-1], -1)


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "quantise":
        rows, cols = case["rows"], case["cols"]
        # normal values, each row at its own size, as weights' output channels and hidden states have
        size = torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))
        state["x"] = (torch.randn((rows, cols), generator=g, device="cuda") * size).to(dtype)
        if own:
            width = cols // 2 if case["format"] == "fp4" else cols
            state["codes"] = torch.empty((rows, width), dtype=torch.uint8, device="cuda")
            state["scales"] = torch.empty((rows, cols // BLOCK), dtype=torch.uint8, device="cuda")
            state["values"] = torch.empty((rows, cols), dtype=dtype, device="cuda")
        return state
    if case["op"] == "norm":
        T, d = case["tokens"], case["hidden"]
        state["x"] = torch.randn((T, d), generator=g, device="cuda").to(dtype)
        state["residual"] = (3 * torch.randn((T, d), generator=g, device="cuda")).to(dtype) if case["residual"] else None
        state["gamma"] = (1 + 0.1 * torch.randn((d,), generator=g, device="cuda")).to(dtype)
        if own:
            import sparse_mixture_experts_04_amd as moe
            width = d // 2 if case["format"] == "fp4" else d
            state["cfg"] = moe.config(T, d, d, 1, 1, -1, case["dtype"])
            state["sum"], state["y"] = torch.empty_like(state["x"]), torch.empty_like(state["x"])
            state["codes"] = torch.empty((T, width), dtype=torch.uint8, device="cuda")
            state["scales"] = torch.empty((T, d // BLOCK), dtype=torch.uint8, device="cuda")
            state["values"] = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
        return state
    T, d, F, E, k, form = (case[n] for n in ("tokens", "hidden", "inner", "experts", "topk", "format"))
    state["xq"], state["xs"] = _random_mx(g, (T, d), 1.0, form)
    state["w1q"], state["w1s"] = _random_mx(g, (E, F, d), 1.0 / math.sqrt(d), "fp4")
    state["w2q"], state["w2s"] = _random_mx(g, (E, d, F), 1.0 / math.sqrt(F), "fp4")
    # the dispatch of the batch: k distinct experts for each token, rows in order of (expert, token, slot)
    bias = 0.3 * torch.randn((E,), generator=g, device="cuda")
    ids = torch.topk(torch.randn((T, E), generator=g, device="cuda") + bias, k, dim=1).indices.reshape(-1)
    perm = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    state["perm"] = perm.to(torch.int32)
    state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    # the same dispatch as a plan for batched products: which row stands in which place of its expert
    active = counts.nonzero().reshape(-1)
    state["active"], state["most"] = active, int(counts.max())
    where = torch.zeros(E, dtype=torch.int64, device="cuda")
    where[active] = torch.arange(active.numel(), device="cuda")
    start = counts.cumsum(0) - counts
    state["place"] = where[ids[perm]] * state["most"] + torch.arange(T * k, device="cuda") - start[ids[perm]]
    state["token"] = perm // k
    if own:
        import sparse_mixture_experts_04_amd as moe
        state["cfg"] = moe.config(T, d, F, E, k, -1, case["dtype"])
        state["y"] = torch.empty((T * k, d), dtype=dtype, device="cuda")
        size = moe.moe_workspace_size(state["cfg"], moe.MOE_OP_EXPERT_FFN_MX)
        state["ws"] = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    return state


# ---- plain forms, in 32 bits

def _two(e):
    """2^e in 32 bits for whole e in [-127, 127], from its bits: a power function need not be exact."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x, form):
    """Element values (before the scale) [rows, cols / 32, 32] and scale exponents [rows, cols / 32] of x [rows, cols]."""
    v = x.view(x.shape[0], -1, BLOCK)
    amax = v.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - EMAX[form], -127).clamp(-127, 127)
    s = v * _two(-e).unsqueeze(-1)
    low, digits = (0, 1) if form == "fp4" else (-6, 3)
    unit = torch.frexp(s).exponent.sub_(1).clamp_(min=low).sub_(digits)   # the last place of each element
    q = (torch.round(s * _two(-unit)) * _two(unit)).clamp_(-TOP[form], TOP[form])
    return q.view(x.shape[0], -1), e


def _scaled(q, e):
    return (q.view(*e.shape, BLOCK) * _two(e).unsqueeze(-1)).view(*q.shape)


def _decode(codes, scales, form):
    """The 32-bit values of code bytes [..., cols or cols / 2] and scale bytes [..., cols / 32]."""
    if form == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        nibble = torch.cat([half, -half])
        byte = torch.arange(256, device=codes.device)
        pair = torch.stack([nibble[byte & 15], nibble[byte >> 4]], dim=-1)
        v = pair.index_select(0, codes.reshape(-1).int()).view(*codes.shape[:-1], -1)
    unit = _two(scales.int() - 127)
    return (v.view(*scales.shape, BLOCK) * unit.unsqueeze(-1)).view(*v.shape)


def _plain(state):
    case = state["case"]
    form, dtype = case["format"], DTYPES[case["dtype"]]
    if case["op"] == "quantise":
        return _scaled(*_quantise(state["x"].float(), form)).to(dtype)
    if case["op"] == "norm":
        s = state["x"].float()
        if state["residual"] is not None:
            s = s + state["residual"].float()
        n = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS) * state["gamma"].float()
        return {"sum": s.to(dtype), "y": n.to(dtype), "values": _scaled(*_quantise(n, form)).to(torch.bfloat16)}
    active, most, place = state["active"], state["most"], state["place"]
    x = _decode(state["xq"], state["xs"], form)
    rows = x.new_zeros((active.numel() * most, x.shape[1]))
    rows[place] = x[state["token"]]
    every = active.numel() == state["w1q"].shape[0]
    pick = (lambda w: w) if every else (lambda w: w[active])
    w = _decode(pick(state["w1q"]), pick(state["w1s"]), "fp4")
    h = torch.bmm(rows.view(active.numel(), most, -1), w.transpose(1, 2))
    del w
    h = 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h)))
    h = _scaled(*_quantise(h.view(-1, h.shape[-1]), form)).view(h.shape)
    w = _decode(pick(state["w2q"]), pick(state["w2s"]), "fp4")
    y = torch.bmm(h, w.transpose(1, 2))
    return y.view(active.numel() * most, -1)[place].to(dtype)


# ---- the package's kernels

def _own(state):
    import sparse_mixture_experts_04_amd as moe

    case = state["case"]
    form = moe.MOE_MXFP4 if case["format"] == "fp4" else moe.MOE_MXFP8
    kind = moe.MOE_BF16 if case["dtype"] == "bf16" else moe.MOE_F32
    if case["op"] == "quantise":
        rows, cols = case["rows"], case["cols"]
        moe.moe_mx_quantize(kind, form, rows, cols, state["x"], state["codes"], state["scales"])
        moe.moe_mx_dequantize(kind, form, rows, cols, state["codes"], state["scales"], state["values"])
        return state["values"]
    if case["op"] == "norm":
        T, d = case["tokens"], case["hidden"]
        moe.moe_add_rmsnorm(state["cfg"], state["x"], state["residual"], state["gamma"], EPS, state["sum"], state["y"],
                            form, state["codes"], state["scales"])
        moe.moe_mx_dequantize(moe.MOE_BF16, form, T, d, state["codes"], state["scales"], state["values"])
        return {"sum": state["sum"], "y": state["y"], "values": state["values"]}
    moe.moe_expert_ffn_mx(state["cfg"], form, state["xq"], state["xs"], state["perm"], state["offsets"], state["w1q"],
                          state["w1s"], state["w2q"], state["w2s"], state["y"], state["ws"])
    return state["y"]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    width = 0.5 if case["format"] == "fp4" else 1.0
    size = 2 if case["dtype"] == "bf16" else 4
    mx = width + 1 / BLOCK
    if case["op"] == "quantise":  # the values read, the codes and scales written and read back, the values written
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * size + 2 * mx), "flops": 0}
    if case["op"] == "norm":
        n = case["tokens"] * case["hidden"]
        return {"bytes": n * ((4 if case["residual"] else 3) * size + 2 * mx + 2) + case["hidden"] * size, "flops": 0}
    T, d, F, E, k = (case[x] for x in ("tokens", "hidden", "inner", "experts", "topk"))
    active = E * (1 - (1 - k / E) ** T)  # experts that some token goes to, on average
    weights = 2 * active * F * d * (0.5 + 1 / BLOCK)
    return {"bytes": T * d * mx + weights + T * k * (d * size + 4) + 4 * (E + 1), "flops": 4.0 * T * k * F * d}


# ---- the definition in 64 bits

def _power(e):
    """2^e in 64 bits, exactly, for whole e held as 64-bit floating numbers."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_mx(v, form):
    """v (64 bits) [..., n * 32] -> the values of its MX form."""
    b = v.reshape(-1, BLOCK)
    top = b.abs().max(dim=1, keepdim=True).values
    exponent = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    # log2 may round up to a whole number just below a power of two
    exponent = torch.where(_power(exponent) > top, exponent - 1, exponent)
    exponent = torch.where(_power(exponent + 1) <= top, exponent + 1, exponent)
    shared = torch.where(top > 0, exponent - (8 if form == "fp8" else 2), torch.full_like(exponent, -127.0)).clamp(-127, 127)
    scale = _power(shared)
    # every non-negative value of the element type, in order: the position is the code
    if form == "fp4":
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    else:
        code = torch.arange(127, device=v.device)
        field, part = code // 8, (code % 8).double()
        table = torch.where(field > 0, (1 + part / 8) * _power(field - 7), part / 8 * 2.0 ** -6)
    a = (b.abs() / scale).clamp(max=float(table[-1]))
    above = torch.searchsorted(table, a).clamp(max=table.numel() - 1)   # first code at or above
    below = (above - 1).clamp(min=0)
    up, down = table[above] - a, a - table[below]
    take = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    return (torch.copysign(table[take], b) * scale).reshape(v.shape)


def _exact_read(codes, scales, form):
    c = codes.to(torch.int64)
    if form == "fp4":
        c = torch.stack([c % 16, c // 16], dim=-1).flatten(-2)
        sign, field, part = c // 8, (c // 2) % 4, (c % 2).double()
        mag = torch.where(field > 0, (1 + part / 2) * _power(field - 1), part / 2)
    else:
        sign, field, part = c // 128, (c // 8) % 16, (c % 8).double()
        mag = torch.where(field > 0, (1 + part / 8) * _power(field - 7), part / 8 * 2.0 ** -6)
    scale = _power(scales.to(torch.int64) - 127).repeat_interleave(BLOCK, dim=-1)
    return torch.where(sign > 0, -mag, mag) * scale


def exact(case, seed):
    state = prepare(case, seed)
    form = case["format"]
    if case["op"] == "quantise":
        step = max(1, (1 << 26) // case["cols"])
        return torch.cat([_exact_mx(part.double(), form).float() for part in state["x"].split(step)])  # exact in 32 bits
    if case["op"] == "norm":
        s = state["x"].double()
        if state["residual"] is not None:
            s = s + state["residual"].double()
        n = s / torch.sqrt((s * s).sum(-1, keepdim=True) / case["hidden"] + EPS) * state["gamma"].double()
        return {"sum": s, "y": n, "values": _exact_mx(n, form)}
    y = torch.zeros((case["tokens"] * case["topk"], case["hidden"]), dtype=torch.float64, device="cuda")
    ends = state["offsets"].tolist()
    for e in range(case["experts"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        source = state["perm"][a:b].long() // case["topk"]
        x = _exact_read(state["xq"][source], state["xs"][source], form)
        h = x @ _exact_read(state["w1q"][e], state["w1s"][e], "fp4").t()
        h = h / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)))
        y[a:b] = _exact_mx(h, form) @ _exact_read(state["w2q"][e], state["w2s"][e], "fp4").t()
    return y
