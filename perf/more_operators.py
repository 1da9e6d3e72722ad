"""What is timed of the 8-bit path in front of and inside a mixture-of-experts layer: the norm that ends in
8 bits, quantisation, and products of 8-bit operands with a scale for each block of 128.

Each case is one call of an operator at sizes that serving meets.  Where `own` is false, `run` computes
the operator from elementary torch operations; where it is true, it calls the library.

Format: e4m3 codes, one byte a value, rows of cols rounded up to 16 bytes, and one fp32 scale for every block:
128 values of a row (activations), or 128 x 128 values (weights); blocks at a row's or matrix's end are cut.
A block's scale is its largest magnitude / 448 ("amax") or the smallest power of two that is no less
("pow2"), at least 2^-126.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = 2.0 ** -126


# ---- cases ------------------------------------------------------------------------------------
def _norm(rows, cols, dtype, residual, values, pad=0, weight="same"):
    return {"op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual, "values": values,
            "pad": pad, "weight": weight}


def _quantize(rows, cols, dtype, block_rows, rule, pad=0):
    return {"op": "quantize", "rows": rows, "cols": cols, "dtype": dtype, "block_rows": block_rows, "rule": rule,
            "pad": pad}


def _linear(m, n, k, out):
    return {"op": "linear", "m": m, "n": n, "k": k, "out": out}


def _experts(part, n, experts, top_k, hidden, inter, routing, out):
    return {"op": "experts", "part": part, "n": n, "experts": experts, "top_k": top_k, "hidden": hidden,
            "inter": inter, "routing": routing, "out": out}


def listed():
    named = [
        # one token of a decode step in front of a layer: sum for the residual stream, 8 bits for the
        # experts, the normed values for the router
        ("norm_one_token", _norm(1, 4096, "bf16", True, True)),
        # a ragged prefill chunk read from a wider buffer, first layer (no residual yet), fp32 activations, a last
        # block that is not full
        ("norm_ragged", _norm(683, 8136, "fp32", False, False, 24)),
        # a long prefill batch
        ("norm_prefill", _norm(16384, 4096, "bf16", True, True)),
        # activations of a prefill chunk that no norm has quantised, scales held to powers of two
        ("quantize_chunk", _quantize(1024, 4096, "bf16", 1, "pow2")),
        # a weight matrix brought to 8 bits when a model is loaded
        ("quantize_weight", _quantize(8192, 8136, "fp32", 128, "amax", 56)),
        # a dense layer's step for one token
        ("linear_one_token", _linear(1, 4096, 4096, "bf16")),
        # a ragged batch against a matrix whose sizes are no tile's or block's multiple
        ("linear_ragged", _linear(683, 2056, 4064, "fp32")),
        # a prefill batch through a large dense layer
        ("linear_prefill", _linear(4096, 8192, 8192, "bf16")),
        # one token through the fused gate and up matrices of its experts, h left in 8 bits for the down pass
        ("experts_one_token", _experts("gate_up", 1, 256, 6, 4096, 2048, "uniform", "e4m3")),
        # a decode batch, skewed routing, down matrices
        ("experts_decode_down", _experts("down", 32, 256, 6, 4096, 2048, "zipf", "fp32")),
        # a prefill chunk, every expert woken
        ("experts_chunk", _experts("gate_up", 1024, 256, 6, 4096, 2048, "uniform", "e4m3")),
        # a long prefill batch, down matrices
        ("experts_prefill_down", _experts("down", 8192, 256, 6, 4096, 2048, "uniform", "bf16")),
    ]
    return [dict(case, name=name) for name, case in named]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "experts"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "norm":
        cols = rng.choice([128 * rng.randint(1, 64), _log(rng, 32, 8192)])
        return _norm(_log(rng, 1, 16384), cols, dtype, rng.random() < 0.6, rng.random() < 0.6, rng.choice([0, 0, 8, 5]),
                     rng.choice(["same", "fp32"]))
    if op == "quantize":
        return _quantize(_log(rng, 1, 8192), _log(rng, 32, 8136), dtype, rng.choice([1, 128]),
                         rng.choice(["amax", "pow2"]), rng.choice([0, 0, 8, 3]))
    if op == "linear":
        k = rng.choice([128 * _log(rng, 1, 64), 16 * _log(rng, 1, 512)])
        return _linear(_log(rng, 1, 8192), _log(rng, 16, 8192), k, rng.choice(["bf16", "fp32"]))
    part = rng.choice(["gate_up", "down"])
    experts = rng.choice([1, 8, 24, 64, 160, 256])
    top_k = rng.randint(1, min(6, experts))
    return _experts(part, _log(rng, 1, 4096), experts, top_k, 128 * rng.randint(1, 32), 128 * rng.randint(1, 16),
                    rng.choice(["uniform", "zipf"]),
                    rng.choice(["bf16", "e4m3"] if part == "gate_up" else ["bf16", "fp32"]))


# ---- inputs -----------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, rows, cols):
    """Hidden states: normal values, a few channels an order of magnitude larger than the rest."""
    x = _randn(g, rows, cols)
    loud = torch.rand(cols, generator=g, device=DEV) < 0.01
    return torch.where(loud, 12.0 * x, x)


def _blocks(cols):
    return (cols + 127) // 128


def _packed(v, block_rows):
    """Codes (uint8) and scales of finite values in fp32, cols a multiple of 16."""
    rows, cols = v.shape
    scales = torch.empty((rows + block_rows - 1) // block_rows, _blocks(cols), device=DEV)
    codes = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    full = cols // 128 * 128
    for c0, c1 in ((0, full), (full, cols)):
        for r0, r1 in ((0, rows // block_rows * block_rows), (rows // block_rows * block_rows, rows)):
            if c0 == c1 or r0 == r1:
                continue
            high, wide = min(block_rows, r1 - r0), min(128, c1 - c0)
            part = v[r0:r1, c0:c1].reshape((r1 - r0) // high, high, (c1 - c0) // wide, wide)
            s = (part.abs().amax(dim=(1, 3)) / 448.0).clamp_min(TINY)
            scales[r0 // block_rows:r0 // block_rows + s.shape[0], c0 // 128:c0 // 128 + s.shape[1]] = s
            code = (part / s[:, None, :, None]).to(F8).view(torch.uint8)
            codes[r0:r1, c0:c1] = code.reshape(r1 - r0, c1 - c0)
    return codes, scales


def _packed_normal(g, matrices, rows, cols, std):
    """Codes and 128 x 128 scales of matrices of normal weights, a piece at a time."""
    codes = torch.empty(matrices, rows, cols, dtype=torch.uint8, device=DEV)
    scales = torch.empty(matrices, _blocks(rows), _blocks(cols), device=DEV)
    for i in range(matrices):
        codes[i], scales[i] = _packed(_randn(g, rows, cols).mul_(std), 128)
    return codes, scales


def _routes(g, case):
    """A batch's expert choices and their bins: (offsets [E + 1], pair ids in expert order)."""
    n, experts, k = case["n"], case["experts"], case["top_k"]
    logits = -torch.log(-torch.log(torch.rand(n, experts, generator=g, device=DEV).clamp(1e-12, 1.0 - 1e-7)))
    if case["routing"] == "zipf":
        rank = torch.randperm(experts, generator=g, device=DEV) + 1
        logits = logits - 1.1 * torch.log(rank.float())
    flat = logits.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(flat, stable=True).indices.to(torch.int32)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=experts), 0).to(torch.int32)
    return offsets, order


class _Plan:
    """A plan of the library, destroyed with its owner."""

    def __init__(self, lib, *desc):
        self.lib = lib
        self.handle = lib.qtip_moe_plan(lib.make_desc(*desc), torch.cuda.current_device())

    def __del__(self):
        self.lib.qtip_moe_plan_destroy(self.handle)


def _library():
    import trellis_quantized_moe_expert_amd as lib
    return lib


def _expert_shape(case):
    """(output rows of one matrix, its inputs, matrices) of an expert pass."""
    if case["part"] == "gate_up":
        return case["inter"], case["hidden"], 2
    return case["hidden"], case["inter"], 1


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] in ("norm", "quantize"):
        rows, cols, t = case["rows"], case["cols"], TYPES[case["dtype"]]
        st["x"] = _activations(g, rows, cols + case["pad"]).to(t)[:, :cols]
        high = case.get("block_rows", 1)
        st["codes"] = torch.empty(rows, (cols + 15) // 16 * 16, dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty((rows + high - 1) // high, _blocks(cols), device=DEV)
    if case["op"] == "norm":
        st["w_t"] = (1.0 + 0.1 * _randn(g, cols)).to(torch.float32 if case["weight"] == "fp32" else t)
        st["res"] = 3.0 * _activations(g, rows, cols) if case["residual"] else None
        st["res"] = st["res"].to(t) if case["residual"] else None
        st["sum"] = torch.empty(rows, cols, dtype=t, device=DEV) if case["residual"] else None
        st["vals"] = torch.empty(rows, cols, dtype=t, device=DEV) if case["values"] else None
    elif case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        st["a_codes"], st["a_scales"] = _packed(_activations(g, m, k), 1)
        w = _packed_normal(g, 1, n, k, 1.0 / math.sqrt(k))
        st["w_codes"], st["w_scales"] = w[0][0], w[1][0]
        st["y"] = torch.empty(m, n, dtype=TYPES[case["out"]], device=DEV)
    elif case["op"] == "experts":
        n, experts, k = case["n"], case["experts"], case["top_k"]
        rows, cols, halves = _expert_shape(case)
        st["offsets"], st["sorted"] = _routes(g, case)
        st["a_codes"], st["a_scales"] = _packed(_activations(g, n if halves == 2 else n * k, cols), 1)
        st["weights"] = [_packed_normal(g, experts, rows, cols, 1.0 / math.sqrt(cols)) for _ in range(halves)]
        if case["out"] == "e4m3":
            st["y"] = torch.empty(n * k, rows, dtype=torch.uint8, device=DEV)
            st["y_scales"] = torch.empty(n * k, rows // 128, device=DEV)
        else:
            st["y"] = torch.empty(n * k, rows, dtype=TYPES[case["out"]], device=DEV)
            st["y_scales"] = None
        if own:
            lib = _library()
            st["plan"] = _Plan(lib, experts, k, case["hidden"], case["inter"], n)
            names = ("gate", "up") if halves == 2 else ("down",)
            st["w"] = lib.make_f8_weights(**{f"{what}_{name}": pair[j] for name, pair in zip(names, st["weights"])
                                             for j, what in enumerate(("codes", "scales"))})
    return st


# ---- the plain forms --------------------------------------------------------------------------
def _power(e):
    """2^e in 64 bits, put together from its bits: exact wherever it runs."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise_plain(v, block_rows, rule):
    """(codes as e4m3 values [rows][cols rounded up to 16], scales) of rows of finite values."""
    rows, cols = v.shape
    high, wide = (rows + block_rows - 1) // block_rows * block_rows, _blocks(cols) * 128
    v = v.float()
    if (high, wide) != (rows, cols):
        v = torch.nn.functional.pad(v, (0, wide - cols, 0, high - rows))
    v = v.reshape(high // block_rows, block_rows, wide // 128, 128)
    top = v.abs().amax(dim=(1, 3))
    scale = (top.double() / 448.0).float()    # in 32 bits a division by a number becomes a product with its inverse
    if rule == "pow2":
        # 448 = 1.75 2^8: the power of two is 2^-8 times that of the largest value, twice where its mantissa passes 1.75
        mant, exp = torch.frexp(top)
        scale = torch.where(top > 0, _power(exp - 9 + (mant > 0.875).int()).float(), scale)
    scale = scale.clamp_min(TINY)
    # in 64 bits: a quotient next to the border between two codes
    ratio = v.double() / scale.double()[:, None, :, None]
    step = torch.frexp(ratio).exponent.clamp_min(-5) - 4
    code = (torch.round(ratio * _power(-step)) * _power(step)).to(F8)
    code = code.reshape(high, wide)[:rows, :(cols + 15) // 16 * 16]
    return code.contiguous(), scale


def _norm_plain(st):
    h = st["x"].float()
    if st["res"] is not None:
        h = (h + st["res"].float()).to(st["x"].dtype)
    total = h
    h = h.float()
    y = h * (1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + 1e-6)) * st["w_t"].float()
    codes, scales = _quantise_plain(y, 1, "amax")
    return {"codes": codes, "scales": scales, "sum": total if st["res"] is not None else None,
            "values": y.to(st["x"].dtype) if st["values"] else None}


def _spread(scales, rows, cols, block_rows):
    """A scale for every value."""
    return scales.repeat_interleave(block_rows, dim=0)[:rows].repeat_interleave(128, dim=1)[:, :cols]


def _values(codes, scales, block_rows):
    """The numbers that codes and scales stand for, in fp32."""
    return codes.view(F8).float() * _spread(scales, codes.shape[0], codes.shape[1], block_rows)


def _linear_plain(st):
    y = _values(st["a_codes"], st["a_scales"], 1) @ _values(st["w_codes"], st["w_scales"], 128).t()
    return y.to(TYPES[st["out"]])


def _experts_plain(st):
    """The pairs' products with their experts' matrices, rows in pair order."""
    rows, _, halves = _expert_shape(st)
    act = _values(st["a_codes"], st["a_scales"], 1)
    offsets = st["offsets"].tolist()
    order = st["sorted"].long()
    y = torch.empty(order.numel(), rows, device=DEV)
    for e in range(st["experts"]):
        pairs = order[offsets[e]:offsets[e + 1]]
        if pairs.numel() == 0:
            continue
        x = act[pairs // st["top_k"] if halves == 2 else pairs]
        one = [x @ _values(c[e], s[e], 128).t() for c, s in st["weights"]]
        y[pairs] = one[0] / (1.0 + torch.exp(-one[0])) * one[1] if halves == 2 else one[0]
    if st["out"] == "e4m3":
        return _quantise_plain(y, 1, "amax")
    return y.to(TYPES[st["out"]])


# ---- one pass ---------------------------------------------------------------------------------
def run(st):
    if not own:
        if st["op"] == "norm":
            return _norm_plain(st)
        if st["op"] == "quantize":
            return _quantise_plain(st["x"], st["block_rows"], st["rule"])
        return _linear_plain(st) if st["op"] == "linear" else _experts_plain(st)
    lib = _library()
    types = {"bf16": lib.QTIP_F8_BF16, "fp16": lib.QTIP_F8_F16, "fp32": lib.QTIP_F8_F32}
    outs = {"bf16": lib.QTIP_OUT_BF16, "fp32": lib.QTIP_OUT_F32, "e4m3": lib.QTIP_OUT_E4M3}
    rules = {"amax": lib.QTIP_F8_SCALE_AMAX, "pow2": lib.QTIP_F8_SCALE_POW2}
    if st["op"] == "norm":
        x = st["x"]
        lib.qtip_f8_rms_norm(x, types[st["dtype"]], x.shape[0], x.shape[1], x.stride(0), st["res"], x.shape[1], st["sum"],
                             st["w_t"], types["fp32" if st["weight"] == "fp32" else st["dtype"]], 1e-6,
                             rules["amax"], st["codes"], st["scales"], st["vals"])
        return {"codes": st["codes"].view(F8), "scales": st["scales"], "sum": st["sum"], "values": st["vals"]}
    if st["op"] == "quantize":
        x = st["x"]
        lib.qtip_f8_quantize(x, types[st["dtype"]], x.shape[0], x.shape[1], x.stride(0), st["block_rows"],
                             rules[st["rule"]], st["codes"], st["scales"])
        return st["codes"].view(F8), st["scales"]
    if st["op"] == "linear":
        lib.qtip_f8_matmul(st["a_codes"], st["a_scales"], st["m"], st["w_codes"], st["w_scales"], st["n"], st["k"],
                           st["y"], outs[st["out"]])
        return st["y"]
    part = lib.QTIP_F8_PASS_GATE_UP if st["part"] == "gate_up" else lib.QTIP_F8_PASS_DOWN
    lib.qtip_f8_expert_matmul(st["plan"].handle, part, st["w"], st["a_codes"], st["a_scales"], st["offsets"],
                              st["sorted"], st["n"], st["y"], outs[st["out"]], st["y_scales"])
    return (st["y"].view(F8), st["y_scales"]) if st["out"] == "e4m3" else st["y"]


# ---- what a pass cannot do without ------------------------------------------------------------
def work(case):
    if case["op"] in ("norm", "quantize"):
        rows, cols = case["rows"], case["cols"]
        size = 4 if case["dtype"] == "fp32" else 2
        high = case.get("block_rows", 1)
        out = rows * ((cols + 15) // 16 * 16) + 4 * ((rows + high - 1) // high) * _blocks(cols)
        if case["op"] == "quantize":
            return {"bytes": rows * cols * size + out, "flops": 3 * rows * cols}
        more = 2 * case["residual"] + case["values"]
        return {"bytes": rows * cols * size * (1 + more) + out + cols * (4 if case["weight"] == "fp32" else size),
                "flops": (7 + case["residual"]) * rows * cols}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * (k + 4 * _blocks(k)) + n * k + 4 * _blocks(n) * _blocks(k)
                + m * n * (4 if case["out"] == "fp32" else 2), "flops": 2 * m * n * k}
    rows, cols, halves = _expert_shape(case)
    n, experts, k = case["n"], case["experts"], case["top_k"]
    pairs = n * k
    # experts that the batch wakes: all that the closed form of uniform routing expects
    woken = max(1.0, experts * (1.0 - (1.0 - k / experts) ** n))
    read = (n if halves == 2 else pairs) * (cols + cols // 32)
    size = {"bf16": 2.0, "fp32": 4.0, "e4m3": 1.0 + 4.0 / 128}[case["out"]]
    return {"bytes": int(woken * halves * rows * cols * (1.0 + 4.0 / 16384) + pairs * rows * size) + read
            + 4 * (pairs + experts + 1), "flops": 2 * halves * pairs * rows * cols}


# ---- the definitions in 64 bits ---------------------------------------------------------------
def _grid():
    """The magnitudes of the codes 0 .. 126, from the format: four bits of exponent (bias 7), three of mantissa."""
    values = [(8 + c % 8) * 2.0 ** (c // 8 - 10) if c >= 8 else c * 2.0 ** -9 for c in range(127)]
    return torch.tensor(values, dtype=torch.float64, device=DEV)


def _exact_quantise(v, block_rows, rule):
    """Every block's scale, and every code the nearest on the grid (a tie: the even code)."""
    rows, cols = v.shape
    grid = _grid()
    middle = (grid[1:] + grid[:-1]) / 2
    codes = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.uint8, device=DEV)
    scales = torch.empty(-(-rows // block_rows), _blocks(cols), dtype=torch.float32, device=DEV)
    step = 128
    for r in range(0, rows, step):
        part = v[r:r + step].double()
        high = part.shape[0]
        top = part.abs()
        if block_rows > 1:
            top = top.amax(dim=0, keepdim=True)
        top = torch.stack([t.amax(dim=1) for t in top.split(128, dim=1)], dim=1)
        if rule == "amax":
            s = (top / 448.0).float().double()
        else:
            s = (top / 448.0).view(torch.int64)        # its exponent alone: the power of two below
            s = ((s >> 52) << 52).view(torch.float64)
            s = torch.where(448.0 * s < top, 2.0 * s, s)
        s = s.clamp_min(TINY)
        scales[r // block_rows:r // block_rows + s.shape[0]] = s.float()
        ratio = part.abs() / s.repeat_interleave(128, dim=1)[:, :cols]
        down = torch.bucketize(ratio, middle)          # middles strictly below the ratio
        tie = ratio == middle[down.clamp_max(125)]
        code = torch.where(tie & (down % 2 == 1), down + 1, down)
        codes[r:r + high, :cols] = (code + 128 * torch.signbit(part)).to(torch.uint8)
    return codes.view(F8), scales


def _exact_spread(codes, scales, block_rows):
    c = codes.long()
    v = torch.where(c >= 128, -1.0, 1.0).double() * _grid()[c % 128]
    r = torch.arange(c.shape[0], device=DEV) // block_rows
    b = torch.arange(c.shape[1], device=DEV) // 128
    return v * scales.double()[r][:, b]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantise(st["x"], case["block_rows"], case["rule"])
    if case["op"] == "norm":
        parts = []
        for r in range(0, case["rows"], 1024):
            h = st["x"][r:r + 1024].double()
            if case["residual"]:
                h = (h + st["res"][r:r + 1024].double()).to(st["x"].dtype).double()
            y = h / (h.square().sum(dim=1, keepdim=True) / case["cols"] + 1e-6).sqrt() * st["w_t"].double()
            parts.append((*_exact_quantise(y, 1, "amax"), h, y))
        codes, scales, total, y = (torch.cat([p[i] for p in parts]) for i in range(4))
        return {"codes": codes, "scales": scales, "sum": total if case["residual"] else None,
                "values": y if case["values"] else None}
    if case["op"] == "linear":
        a = _exact_spread(st["a_codes"], st["a_scales"], 1)
        # block rows of the weights at a time
        return torch.cat([a @ _exact_spread(st["w_codes"][r:r + 1024], st["w_scales"][r // 128:r // 128 + 8],
                                            128).T.contiguous() for r in range(0, case["n"], 1024)], dim=1)
    rows, _, halves = _expert_shape(case)
    owner = torch.empty(case["n"] * case["top_k"], dtype=torch.long, device=DEV)
    counts = (st["offsets"][1:] - st["offsets"][:-1]).long()
    owner[st["sorted"].long()] = torch.repeat_interleave(torch.arange(case["experts"], device=DEV), counts)
    act = _exact_spread(st["a_codes"], st["a_scales"], 1)
    if halves == 2:
        act = act.repeat_interleave(case["top_k"], dim=0)
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device=DEV)
    for e in owner.unique().tolist():
        mine = (owner == e).nonzero().flatten()
        prod = [act[mine] @ _exact_spread(c[e], s[e], 128).T.contiguous() for c, s in st["weights"]]
        y[mine] = prod[0] * torch.sigmoid(prod[0]) * prod[1] if halves == 2 else prod[0]
    return _exact_quantise(y, 1, "amax") if case["out"] == "e4m3" else y
