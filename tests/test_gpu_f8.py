"""e4m3 on the GPU: quantisation against the oracle bit for bit; the norm and the products against float64 within
bounds derived from their sums (f8_util) and the output's rounding."""
import numpy as np
import pytest

import trellis_quantized_moe_expert_amd as q
from f8_util import (OUT, RULE, TYPE, check_codes, dtype_of, eight_bound, norm_bound, packed, quantise, rounded, same, sum_bound,
                     within)
from gpu_util import say
from mx_util import bins_of
from oracle import f8, mx

pytestmark = pytest.mark.gpu


# ---- quantisation -----------------------------------------------------------------------------
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rule", ["amax", "pow2"])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 128, 0), (3, 129, 0), (2, 127, 5), (5, 100, 0), (4, 4096, 0),
                                           (129, 256, 8), (130, 650, 3), (300, 17, 0), (257, 1000, 24)])
def test_quantise_matches_the_oracle(rows, cols, pad, kind, rule, block_rows):
    import torch
    say(f"quantise {rows}x{cols} pad {pad} {kind} {rule} blocks of {block_rows} rows")
    g = torch.Generator().manual_seed(rows * 10007 + cols)
    wide = torch.randn(rows, cols + pad, generator=g) * torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g).float())
    x = wide.to(dtype_of(kind)).cuda()[:, :cols]
    same(quantise(x, kind, rule, block_rows), f8.quantise(x.cpu().double().numpy(), rule, block_rows))


@pytest.mark.parametrize("rule", ["amax", "pow2"])
def test_quantise_next_to_the_borders(rule):
    # fp32 numbers on and next to every border between two codes, under scales of many mantissas
    import torch
    say(f"quantise borders {rule}")
    rng = np.random.default_rng(5)
    middle = ((f8.GRID[1:] + f8.GRID[:-1]) / 2)
    rows = []
    for amax in np.exp2(rng.uniform(-100, 100, 200)).astype(np.float32):
        s = f8.scale_of(amax, rule)
        near = (middle * s).astype(np.float32)
        step = rng.integers(-3, 4, near.shape, dtype=np.int32)
        near = (near.view(np.int32) + step).view(np.float32)
        row = np.concatenate([np.minimum(near, amax), [amax, -amax / 3]]).astype(np.float32)
        rows.append(np.where(rng.random(128) < 0.5, row, -row))
    x = torch.from_numpy(np.array(rows, np.float32)).cuda()
    same(quantise(x, "fp32", rule), f8.quantise(x.cpu().double().numpy(), rule))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_sources_at_any_elements_address(kind):
    import torch
    say(f"quantise and norm from odd addresses {kind}")
    g = torch.Generator().manual_seed(11)
    flat = torch.randn(3000, generator=g).to(dtype_of(kind)).cuda()
    for at in (1, 3, 5):
        x = flat[at:at + 5 * 301].as_strided((5, 270), (301, 1), at)
        same(quantise(x, kind, "amax"), f8.quantise(x.cpu().double().numpy(), "amax"))
        w = flat[at + 1600:at + 1600 + 270]
        res = flat[at + 1:].as_strided((5, 270), (280, 1), at + 1)
        check_norm(x, kind, res, w, kind, 1e-6)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rule", ["amax", "pow2"])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_quantise_extremes(kind, rule, block_rows):
    # powers of two over the type's whole range, subnormal ones among them, zeros, infinities, NaN
    import torch
    say(f"quantise extremes {kind} {rule} {block_rows}")
    t = dtype_of(kind)
    info = torch.finfo(t)
    low = int(np.log2(info.smallest_normal)) - (10 if kind == "fp16" else 7 if kind == "bf16" else 23)
    high = int(np.floor(np.log2(info.max)))
    x = torch.zeros(high - low + 6, 130)
    for i, e in enumerate(range(low, high + 1)):
        x[i, 3], x[i, 7], x[i, 129] = 2.0 ** e, -(1.9 * 2.0 ** max(e - 2, low)), 2.0 ** max(e - 4, low)
    x = x.to(t)
    n = high - low + 1
    x[n] = info.max
    x[n + 1, 9] = float("inf")
    x[n + 2, 129] = float("nan")
    x[n + 3, 0], x[n + 3, 1] = -0.0, info.max
    x = x.repeat_interleave(block_rows, dim=0)[:, :130].cuda()
    same(quantise(x, kind, rule, block_rows), f8.quantise(x.cpu().double().numpy(), rule, block_rows))


def test_quantise_one_row_of_all_columns_there_can_be():
    import torch
    cols, part = 2 ** 31 - 1, 2 ** 14
    say(f"quantise 1x{cols}")
    base = torch.randn(1, part, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    ref = f8.quantise(base.double().numpy(), "amax")
    x = base.cuda().repeat(1, 2 ** 31 // part)[:, :cols]
    codes = torch.full((2 ** 31,), 0xA5, dtype=torch.uint8, device="cuda:0")
    scales = torch.full((2 ** 24,), -7.0, device="cuda:0")
    q.qtip_f8_quantize(x, TYPE["bf16"], 1, cols, cols, 1, RULE["amax"], codes, scales)
    torch.cuda.synchronize()
    want = torch.from_numpy(ref[0][0]).cuda()
    assert all(bool((piece == want).all()) for piece in codes.view(-1, part)[:-1].split(2 ** 13))
    tail = f8.quantise(base[:, :-1].double().numpy(), "amax")
    assert np.array_equal(codes.view(-1, part)[-1].cpu().numpy(), tail[0][0])
    s = scales.view(-1, part // 128).cpu().numpy()
    assert np.all(s[:-1] == ref[1][0]) and np.array_equal(s[-1], tail[1][0])


# ---- norm -------------------------------------------------------------------------------------
def norm(x, kind, res, w, w_kind, eps, rule, with_values=True, in_place=False):
    """codes, scales, sums, values (numpy, floats as float64)."""
    import torch
    rows, cols = x.shape
    dev = dict(device="cuda:0")
    codes = torch.full((rows, -(-cols // 16) * 16), 0xA5, dtype=torch.uint8, **dev)
    scales = torch.full((rows, -(-cols // 128)), -7.0, **dev)
    vals = torch.full((rows, cols), -7.0, dtype=x.dtype, **dev) if with_values else None
    total = None
    if res is not None:
        total = res if in_place else torch.full((rows, res.stride(0)), -7.0, dtype=x.dtype, **dev)[:, :cols]
    q.qtip_f8_rms_norm(x, TYPE[kind], rows, cols, x.stride(0), res, res.stride(0) if res is not None else 0, total, w,
                       TYPE[w_kind], eps, RULE[rule], codes, scales, vals)
    torch.cuda.synchronize()
    f = lambda t: None if t is None else t.cpu().double().numpy()
    return codes.cpu().numpy(), scales.cpu().numpy(), f(total), f(vals)


def check_norm(x, kind, res, w, w_kind, eps, rule="amax", in_place=False):
    h = x.cpu().double().numpy()
    if res is not None:
        h = (x.cpu().double() + res.cpu().double()).to(x.dtype).double().numpy()
    y = f8.rms_norm(h, w.cpu().double().numpy(), eps)
    codes, scales, total, vals = norm(x, kind, res, w, w_kind, eps, rule, in_place=in_place)
    if res is not None:
        assert np.array_equal(total, h)
    lim = norm_bound(x.shape[1]) * np.abs(y)
    within(vals, y, rounded(lim, y, kind))
    if kind == "fp32":                      # the values are what was quantised
        same((codes, scales), f8.quantise(vals, rule))
    elif rule == "amax":
        check_codes(codes, scales, y, lim)


SHAPES = [(1, 1, 0), (1, 128, 0), (3, 100, 3), (5, 129, 0), (2, 4096, 0), (33, 640, 8), (4, 8136, 24), (3, 8200, 0),
          (2, 16384, 0), (2, 20001, 7), (1, 32768, 0), (2, 32776, 0), (1, 70001, 0)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("kind,w_kind", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16"),
                                         ("bf16", "fp16")])
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_norm_matches_float64(rows, cols, pad, kind, w_kind, residual):
    import torch
    say(f"norm {rows}x{cols} pad {pad} {kind} weight {w_kind} residual {residual}")
    g = torch.Generator().manual_seed(rows * 131 + cols)
    r = lambda *s: torch.randn(*s, generator=g)
    x = r(rows, cols + pad).to(dtype_of(kind)).cuda()[:, :cols]
    res = (3 * r(rows, cols + 2 * pad)).to(dtype_of(kind)).cuda()[:, :cols] if residual else None
    w = (1 + 0.2 * r(cols)).to(dtype_of(w_kind)).cuda()
    check_norm(x, kind, res, w, w_kind, 1e-6, "pow2" if kind == "fp32" and rows == 2 else "amax")


@pytest.mark.parametrize("cols", [256, 40000])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_norm_in_place(kind, cols):
    import torch
    say(f"norm in place {kind} {cols}")
    g = torch.Generator().manual_seed(cols)
    x, res = (torch.randn(5, cols + 8, generator=g).to(dtype_of(kind)).cuda() for _ in range(2))
    behind = res[:, cols:].clone()
    w = torch.ones(cols, device="cuda:0")
    check_norm(x[:, :cols], kind, res[:, :cols], w, "fp32", 1e-5, in_place=True)
    assert torch.equal(res[:, cols:], behind)


@pytest.mark.parametrize("cols", [300, 40000])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-21, 1e18, 1e30, 3e38])
def test_norm_of_rows_whose_squares_leave_fp32(size, cols):
    import torch
    say(f"norm of values of {size}, {cols} columns")
    g = torch.Generator().manual_seed(2)
    x = ((torch.rand(3, cols, generator=g) - 0.5) * 2 * size).cuda()
    w = torch.ones(cols, device="cuda:0")
    for eps in (0.0, 1e-6, 1e-37):
        check_norm(x, "fp32", None, w, "fp32", eps)


def test_norm_of_zeros_infinities_and_nan():
    import torch
    say("norm specials")
    x = torch.randn(4, 300, generator=torch.Generator().manual_seed(1))
    x[0], x[1, 7], x[2, 290] = 0.0, float("inf"), float("nan")
    w = torch.ones(300, device="cuda:0")
    codes, scales, _, vals = norm(x.cuda(), "fp32", None, w, "fp32", 1e-6, "amax")
    assert not vals[0].any() and not codes[0].any() and np.all(scales[0] == np.float32(f8.TINY))
    assert np.isnan(vals[1, 7]) and not np.delete(vals[1], 7).any()
    assert np.isnan(scales[1]).tolist() == [True, False, False]
    assert not codes[1, :128].any() and not f8.TABLE[codes[1]].any()            # -0 of negative values, sign kept
    assert np.isnan(vals[2]).all() and np.isnan(scales[2]).all() and not codes[2].any()
    y = f8.rms_norm(x[3:].double().numpy(), np.ones(300), 1e-6)
    within(vals[3:], y, rounded(norm_bound(300) * np.abs(y), y, "fp32"))
    assert np.isnan(norm(torch.zeros(1, 300).cuda(), "fp32", None, w, "fp32", 0.0, "amax")[3]).all()


def test_norm_values_and_codes_do_not_depend_on_each_other():
    import torch
    say("norm without values")
    x = torch.randn(7, 900, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = torch.ones(900, device="cuda:0").bfloat16()
    a = norm(x, "bf16", None, w, "bf16", 1e-6, "amax")
    b = norm(x, "bf16", None, w, "bf16", 1e-6, "amax", with_values=False)
    same(a[:2], b[:2])
    assert b[3] is None


# ---- products ---------------------------------------------------------------------------------
def product(a, w, k, kind):
    import torch
    dev = [torch.from_numpy(t).cuda() for t in (*a, *w)]
    m, n = a[0].shape[0], w[0].shape[0]
    out = torch.full((m, n), -7.0, dtype=dtype_of(kind), device="cuda:0")
    q.qtip_f8_matmul(dev[0], dev[1], m, dev[2], dev[3], n, k, out, OUT[kind])
    torch.cuda.synchronize()
    return out.cpu().double().numpy()


def check_product(a, w, kind):
    k = a[0].shape[1]
    av, wv = f8.decode(*a), f8.decode(*w, 128)
    ref = av @ wv.T
    lim = sum_bound(av, wv, -(-k // 128)) + (eight_bound(av, wv) if kind == "bf16" else 0.0)
    within(product(a, w, k, kind), ref, rounded(lim, ref, kind))


SIZES = [(1, 1, 16), (1, 16, 128), (1, 4096, 512), (2, 17, 144), (3, 100, 560), (15, 33, 1040), (16, 16, 2048),
         (17, 64, 512), (33, 48, 4096), (64, 130, 640), (65, 128, 128), (100, 257, 416), (128, 256, 256),
         (129, 72, 992), (255, 300, 1024), (256, 256, 4096), (300, 513, 160), (513, 1040, 2080), (1, 24, 8192),
         (40, 50, 96), (20, 70, 32), (700, 300, 128), (520, 264, 1184), (4, 136, 4112), (1, 130, 16400),
         (40, 100, 20000), (300, 300, 9008), (330, 2100, 8720)]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_matches_float64(m, n, k, kind):
    say(f"product {m}x{n}x{k} {kind}")
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    check_product(packed(rng, m, k), packed(rng, n, k, 128), kind)


# every tile of the dense product: rows and columns past the tiles' ends, last blocks not full
TILES = [(20, 8200, 96), (130, 4100, 1120), (280, 2056, 96), (290, 2050, 4160), (260, 4104, 2080), (300, 3300, 160),
         (1000, 2056, 160), (1001, 2063, 288), (1030, 3200, 96), (1100, 3207, 544), (4000, 4100, 64),
         (3850, 4351, 352), (683, 2056, 4064), (700, 1800, 608), (700, 1800, 16656)]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", TILES)
def test_large_product_matches_float64(m, n, k, kind):
    say(f"product {m}x{n}x{k} {kind}")
    rng = np.random.default_rng(m * 5 + n + k)
    check_product(packed(rng, m, k), packed(rng, n, k, 128), kind)


@pytest.mark.parametrize("m,n", [(16, 16), (40, 40), (300, 130), (1030, 3200)])
def test_product_one_chunk_at_a_time(m, n):
    # 16 nonzero inputs at a time show any mismatch of codes, scales and lanes: products of few bits, exact sums
    say(f"product chunk by chunk {m}x{n}")
    rng = np.random.default_rng(4)
    k = 400
    for c in range(0, k, 16) if m < 300 else (0, 112, 128, 384):
        a, w = packed(rng, m, k), packed(rng, n, k, 128)
        for codes in (a[0], w[0]):
            small = rng.integers(0x30, 0x40, codes.shape)          # 0.5 .. 1.875: products are multiples of 2^-8
            codes[:] = 0
            codes[:, c:c + 16] = small[:, c:c + 16]
        for scales in (a[1], w[1]):
            scales[:] = np.exp2(rng.integers(-9, 9, scales.shape))
        assert np.array_equal(product(a, w, k, "fp32"), f8.decode(*a) @ f8.decode(*w, 128).T), c


@pytest.mark.parametrize("m,n,k", [(1, 200, 160), (40, 300, 544), (300, 2050, 96), (1000, 2056, 160),
                                   (1030, 3200, 96), (4000, 4100, 64)])
def test_nan_reaches_its_own_outputs_only(m, n, k):
    say(f"product {m}x{n}x{k} with NaN blocks")
    rng = np.random.default_rng(m + n)
    a, w = packed(rng, m, k), packed(rng, n, k, 128)
    before = product(a, w, k, "fp32")
    a[1][m - 1, -1] = np.nan                # the last block of the last row
    w[0][n // 2, k - 1] = 0x7f              # a code
    w[1][-1, 0] = np.nan                    # the first block of the last rows
    after = product(a, w, k, "fp32")
    hit = np.zeros((m, n), bool)
    hit[m - 1] = hit[:, n // 2] = hit[:, (n - 1) // 128 * 128:] = True
    assert np.all(np.isnan(after[hit]))
    assert np.array_equal(after[~hit], before[~hit])


def test_product_scale_extremes():
    say("product scale extremes")
    rng = np.random.default_rng(6)
    check_product(packed(rng, 20, 256, 1, -126, -100), packed(rng, 40, 256, 128, 30, 100), "fp32")
    check_product(packed(rng, 300, 256, 1, 60, 100), packed(rng, 400, 256, 128, -126, -100), "fp32")


# ---- experts ----------------------------------------------------------------------------------
class Experts:
    """A plan, random e4m3 weights (numpy and device) and a routed batch."""

    def __init__(self, seed, n, E, k, H, I, skew=False, holes=0.0, max_tokens=None, out_dtype=q.QTIP_OUT_F32):
        import torch
        rng = np.random.default_rng(seed)
        self.n, self.E, self.k, self.H, self.I = n, E, k, H, I
        self.plan = q.qtip_moe_plan(q.make_desc(E, k, H, I, max_tokens or n, out_dtype=out_dtype), 0)
        self.w = {name: packed(rng, E * rows, cols, 128, -14, -10)
                  for name, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I))}
        self.dev = {name: [torch.from_numpy(t).cuda() for t in v] for name, v in self.w.items()}
        self.weights = q.make_f8_weights(*self.dev["gate"], *self.dev["up"], *self.dev["down"])
        self.idx, self.counts, self.offsets, self.order = bins_of(rng, n, E, k, skew, holes)
        self.x = packed(rng, n, H, 1, -7, -5)
        self.h = packed(rng, n * k, I, 1, -7, -5)

    def run(self, part, kind, offsets=None, order=None):
        """The outputs as float64; of e4m3 (codes, scales)."""
        import torch
        act, width = (self.x, self.I) if part == "gate_up" else (self.h, self.H)
        full = np.full(self.n * self.k, -9, np.int32)
        full[:len(self.order)] = self.order
        dev = [torch.from_numpy(np.ascontiguousarray(t)).cuda()
               for t in (*act, self.offsets if offsets is None else offsets, full if order is None else order)]
        pass_ = q.QTIP_F8_PASS_GATE_UP if part == "gate_up" else q.QTIP_F8_PASS_DOWN
        if kind == "e4m3":
            out = torch.full((self.n * self.k, width), 0xA5, dtype=torch.uint8, device="cuda:0")
            scales = torch.full((self.n * self.k, width // 128), -7.0, device="cuda:0")
            q.qtip_f8_expert_matmul(self.plan, pass_, self.weights, *dev, self.n, out, OUT[kind], scales)
            torch.cuda.synchronize()
            return out.cpu().numpy(), scales.cpu().numpy()
        out = torch.full((self.n * self.k, width), -7.0, dtype=dtype_of(kind), device="cuda:0")
        q.qtip_f8_expert_matmul(self.plan, pass_, self.weights, *dev, self.n, out, OUT[kind])
        torch.cuda.synchronize()
        return out.cpu().double().numpy()

    def matrix(self, name, e):
        rows, cols = (self.H, self.I) if name == "down" else (self.I, self.H)
        codes, scales = self.w[name]
        return f8.decode(codes[e * rows:(e + 1) * rows], scales[e * rows // 128:(e + 1) * rows // 128], 128)

    def reference(self, part, kind):
        """(rows, results, bounds) of each expert with pairs."""
        bound = lambda a, w: sum_bound(a, w, a.shape[1] // 128) + (eight_bound(a, w) if kind == "bf16" else 0.0)
        flat = self.idx.reshape(-1)
        for e in range(self.E):
            pairs = np.flatnonzero(flat == e)
            if not len(pairs):
                continue
            if part == "gate_up":
                a = f8.decode(*self.x)[pairs // self.k]
                g, u = self.matrix("gate", e), self.matrix("up", e)
                gr, ur = a @ g.T, a @ u.T
                ref = mx.silu(gr) * ur
                # silu itself: exp, add, reciprocal and two products in fp32, a few steps of 2^-24 relative
                lim = mx.swiglu_bound(gr, ur, bound(a, g), bound(a, u))
                yield pairs, ref, lim + 8 * 2.0 ** -24 * np.abs(ref)
            else:
                a, d = f8.decode(*self.h)[pairs], self.matrix("down", e)
                yield pairs, a @ d.T, bound(a, d)

    def check(self, part, kind):
        got = self.run(part, kind)
        for pairs, ref, lim in self.reference(part, kind):
            if kind == "e4m3":
                check_codes(got[0][pairs], got[1][pairs], ref, lim)
                continue
            within(got[pairs], ref, rounded(lim, ref, kind))
        left_out = np.flatnonzero(self.idx.reshape(-1) < 0)                  # pairs in no bin: left as they were
        if kind == "e4m3":
            assert np.all(got[0][left_out] == 0xA5) and np.all(got[1][left_out] == -7.0)
            # the fp32 results of the same pass, quantised
            kept = np.flatnonzero(self.idx.reshape(-1) >= 0)
            same((got[0][kept], got[1][kept]), f8.quantise(self.run(part, "fp32")[kept]))
        else:
            assert np.all(got[left_out] == -7.0)

    def close(self):
        q.qtip_moe_plan_destroy(self.plan)


EXPERTS = [
    # n, E, k, H, I, skew, holes
    (1, 8, 2, 256, 128, False, 0.0),
    (1, 1, 1, 128, 128, False, 0.0),
    (3, 64, 6, 512, 384, False, 0.0),
    (9, 16, 4, 1152, 256, False, 0.0),
    (16, 4, 4, 640, 256, False, 0.0),
    (40, 16, 3, 1152, 128, True, 0.0),
    (70, 5, 2, 384, 640, False, 0.3),
    (200, 8, 2, 256, 256, True, 0.1),
    (17, 300, 4, 128, 256, False, 0.0),
    (600, 3, 2, 512, 256, True, 0.0),
    (260, 2, 2, 2048, 128, False, 0.0),
    (1500, 4, 1, 256, 512, True, 0.05),
    (40, 16, 3, 8448, 128, False, 0.0),
    (180, 8, 2, 8320, 128, False, 0.0),
    (300, 4, 2, 8448, 256, False, 0.0),
    (500, 2, 1, 128, 8448, False, 0.0),
]


@pytest.mark.parametrize("part,kind", [("gate_up", "bf16"), ("gate_up", "fp32"), ("gate_up", "e4m3"), ("down", "bf16"),
                                       ("down", "fp32")])
@pytest.mark.parametrize("n,E,k,H,I,skew,holes", EXPERTS)
def test_expert_pass_matches_float64(n, E, k, H, I, skew, holes, part, kind):
    say(f"experts {part} n={n} E={E} k={k} H={H} I={I} skew={skew} holes={holes} {kind}")
    ex = Experts(n * 31 + E, n, E, k, H, I, skew, holes)
    ex.check(part, kind)
    ex.close()


def test_expert_pass_with_no_pair_at_all():
    say("experts without a pair")
    ex = Experts(1, 9, 4, 2, 128, 128, holes=1.0)
    assert np.all(ex.run("gate_up", "bf16") == -7.0)
    assert np.all(ex.run("gate_up", "e4m3")[0] == 0xA5)
    assert np.all(ex.run("down", "fp32") == -7.0)
    ex.close()


@pytest.mark.parametrize("n,part", [(30, "down"), (30, "gate_up"), (3, "gate_up"), (3, "down"), (400, "gate_up")])
def test_expert_pass_holds_bad_bins_to_its_bounds(n, part):
    # the kernels' own checks: offsets outside [0, n k] are held to it, pair ids outside skipped
    say(f"experts bad bins {part} {n}")
    ex = Experts(2, n, 4, 2, 256, 128)
    good = ex.run(part, "fp32")
    order = np.concatenate([ex.order]).astype(np.int32)
    order[[1, 4]] = [2 * n, -2 ** 31]
    got = ex.run(part, "fp32", order=order)
    lost = ex.order[[1, 4]]
    keep = np.setdiff1d(np.arange(2 * n), lost)
    assert np.array_equal(got[keep], good[keep]) and np.all(got[lost] == -7.0)
    offsets = ex.offsets.copy()
    offsets[-1] = 2 ** 31 - 1
    assert np.array_equal(ex.run(part, "fp32", offsets=offsets), good)
    offsets[0] = -5
    assert np.array_equal(ex.run(part, "fp32", offsets=offsets), good)
    ex.close()


def test_a_nan_result_is_a_nan_block():
    say("experts NaN to e4m3")
    ex = Experts(3, 20, 4, 2, 256, 256)
    ex.x[1][5, 1] = np.nan
    codes, scales = ex.run("gate_up", "e4m3")
    assert np.isnan(scales[10:12]).all() and not codes[10:12].any()
    assert not np.isnan(np.delete(scales, [10, 11], axis=0)).any()
    ex.close()


def test_results_do_not_depend_on_the_run():
    say("experts same bits twice")
    ex = Experts(7, 333, 6, 3, 512, 256, skew=True)
    for part in ("gate_up", "down"):
        assert np.array_equal(ex.run(part, "fp32"), ex.run(part, "fp32"))
    ex.close()


@pytest.mark.parametrize("m,n,k", [(1030, 6500, 160), (1500, 4702, 1040), (1153, 5120, 8352), (1281, 5001, 400), (1540, 4099, 1040),
                                   (1154, 5123, 1040), (2500, 4100, 288)])
def test_product_of_wide_tiles_matches_float64(m, n, k):
    say(f"product of 128 x 256 tiles {m}x{n}x{k}")
    rng = np.random.default_rng(m + n + k)
    check_product(packed(rng, m, k, 1, -6, -3), packed(rng, n, k, 128, -6, -3), "bf16")


# every tile of the expert passes, most of them with an expert's last tile cut: pairs an expert, and workgroups enough for it
EXPERT_TILES = [
    # n, E, k, H, I, skew, holes
    (700, 8, 2, 4096, 384, True, 0.1),      # down: 256 x 256 and, fp32, 128 x 128
    (900, 8, 1, 2816, 256, False, 0.0),     # down: 128 x 128
    (900, 8, 1, 2816, 1152, True, 0.05),    # down: 128 x 256 bf16
    (360, 8, 1, 2688, 256, True, 0.0),      # down: 64 x 128
    (40, 16, 3, 2048, 640, True, 0.0),      # down: 32 x 128
    (700, 8, 2, 384, 2048, True, 0.1),      # gate+up: 256 rows bf16, 128 the others
    (900, 8, 1, 256, 2048, False, 0.05),    # gate+up: 128 rows bf16, 64 the others
    (1000, 8, 1, 1152, 2048, True, 0.0),    # the same over more stages
    (360, 8, 1, 640, 2688, True, 0.0),      # gate+up: 64 rows
    (40, 16, 3, 640, 2048, False, 0.0),     # gate+up: 32 rows in two stages
    (1024, 1, 1, 1280, 256, False, 0.0),    # one expert
]


@pytest.mark.parametrize("part,kind", [("gate_up", "bf16"), ("gate_up", "fp32"), ("gate_up", "e4m3"), ("down", "bf16"),
                                       ("down", "fp32")])
@pytest.mark.parametrize("n,E,k,H,I,skew,holes", EXPERT_TILES)
def test_expert_tiles_match_float64(n, E, k, H, I, skew, holes, part, kind):
    say(f"expert tiles {part} n={n} E={E} k={k} H={H} I={I} skew={skew} holes={holes} {kind}")
    ex = Experts(n * 17 + E + H, n, E, k, H, I, skew, holes)
    ex.check(part, kind)
    ex.close()


@pytest.mark.parametrize("n,I", [(900, 2048), (1100, 3328)])
def test_gate_up_tiles_over_more_stages_than_a_register_holds_scales_for(n, I):
    say(f"expert tiles gate_up {n} pairs of one expert, 8448 inputs, {I} outputs")
    ex = Experts(n, n, 1, 1, 8448, I)
    ex.check("gate_up", "bf16")
    ex.close()


@pytest.mark.parametrize("part,H,I", [("down", 4096, 128), ("gate_up", 128, 2048)])
def test_bad_bins_at_the_large_tiles(part, H, I):
    say(f"expert tiles, bad bins {part}")
    n = 700
    ex = Experts(4, n, 8, 2, H, I)
    for kind in ("bf16", "fp32"):
        good = ex.run(part, kind)
        order = ex.order.astype(np.int32)
        order[[1, 400]] = [2 * n, -2 ** 31]
        got, lost = ex.run(part, kind, order=order), ex.order[[1, 400]]
        keep = np.setdiff1d(np.arange(2 * n), lost)
        assert np.array_equal(got[keep], good[keep]) and np.all(got[lost] == -7.0)
        offsets = ex.offsets.copy()
        offsets[0], offsets[-1] = -5, 2 ** 31 - 1
        assert np.array_equal(ex.run(part, kind, offsets=offsets), good)
    ex.close()


def test_norm_of_a_very_long_row_of_equal_values():
    import torch
    say("norm of 2^28 equal values")
    cols, value = 2 ** 28 + 40, float(np.float32(1.1))
    x = torch.full((1, cols), value, device="cuda:0")
    w = torch.ones(cols, device="cuda:0")
    codes = torch.empty(1, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda:0")
    scales = torch.empty(1, -(-cols // 128), device="cuda:0")
    vals = torch.empty_like(x)
    q.qtip_f8_rms_norm(x, TYPE["fp32"], 1, cols, cols, None, 0, None, w, TYPE["fp32"], 1e-6, RULE["amax"], codes, scales, vals)
    y = value / np.sqrt(value * value + 1e-6)
    # eight squares in fp32, the eights in fp64, then as norm_bound: 6 + 16 sums of lanes and waves
    lim = norm_bound(1024 * 8) * y
    assert bool(((vals.double() - y).abs() <= lim).all())
    assert bool((codes[0, :cols] == 0x7e).all()) and not bool(codes[0, cols:].any())
