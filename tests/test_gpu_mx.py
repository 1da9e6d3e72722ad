"""MXFP4 on the GPU: quantisation against the oracle bit for bit, products against float64 within
bounds derived from the sums (mx_util.sum_bound) and the output's rounding."""
import numpy as np
import pytest

import trellis_quantized_moe_expert_amd as q
from gpu_util import say
from mx_util import bins_of, packed, rounded, sum_bound, values
from oracle import mx

pytestmark = pytest.mark.gpu

SRC = {"bf16": q.QTIP_MX_SRC_BF16, "fp16": q.QTIP_MX_SRC_F16, "fp32": q.QTIP_MX_SRC_F32}
RULE = {"floor": q.QTIP_MX_SCALE_FLOOR, "nearest": q.QTIP_MX_SCALE_NEAREST}
OUT = {"bf16": q.QTIP_OUT_BF16, "fp32": q.QTIP_OUT_F32}


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def quantise(x, kind, rule, with_values=True):
    """codes, scales, values (numpy, values as float64) of a 2-D device tensor (rows may be strided)."""
    import torch
    rows, cols = x.shape
    blocks = -(-cols // 32)
    codes = torch.full((rows, blocks * 16), 0xA5, dtype=torch.uint8, device="cuda:0")
    scales = torch.full((rows, blocks), 0xA5, dtype=torch.uint8, device="cuda:0")
    vals = torch.full((rows, cols), -7.0, dtype=x.dtype, device="cuda:0") if with_values else None
    q.qtip_mx_quantize(x, SRC[kind], rows, cols, x.stride(0), RULE[rule], codes, scales, vals)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy(), None if vals is None else vals.cpu().double().numpy()


def check_quantise(x, kind, rule, with_values=True):
    import torch
    got = quantise(x, kind, rule, with_values)
    ref = mx.quantise(x.cpu().double().numpy(), rule)
    assert np.array_equal(got[1], ref[1])
    assert np.array_equal(got[0], ref[0])
    if with_values:
        # exact in the type but past its range: the nearest rule makes 2^128 (fp16: 2^16) of the
        # largest numbers, and the conversion an infinity of that
        want = torch.from_numpy(ref[2]).to(x.dtype).double().numpy()
        assert np.array_equal(want, np.where(np.isinf(want), want, ref[2]), equal_nan=True)
        assert np.array_equal(got[2], want, equal_nan=True)


@pytest.mark.parametrize("rule", ["floor", "nearest"])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 32, 0), (3, 33, 0), (2, 31, 5), (5, 100, 0), (4, 4096, 0),
                                           (7, 256, 8), (9, 160, 3), (17, 96, 0), (2, 1000, 24), (300, 64, 0)])
def test_quantise_matches_the_oracle(rows, cols, pad, kind, rule):
    import torch
    say(f"quantise {rows}x{cols} pad {pad} {kind} {rule}")
    g = torch.Generator().manual_seed(rows * 10007 + cols)
    wide = torch.randn(rows, cols + pad, generator=g) * torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g).float())
    check_quantise(wide.to(dtype_of(kind)).cuda()[:, :cols], kind, rule, with_values=cols != 256)


@pytest.mark.parametrize("cols", [2 ** 31 - 1, 2 ** 31 - 9])
def test_quantise_one_row_of_all_columns_there_can_be(cols):
    # 2^14 values over and over; the last block is not full, its last eight values the last of 31-bit columns
    import torch
    say(f"quantise 1x{cols}")
    part = 2 ** 14
    base = torch.randn(1, part, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    ref = mx.quantise(base.double().numpy(), "nearest")
    x = base.cuda().repeat(1, 2 ** 31 // part)[:, :cols]
    codes = torch.full((1, 2 ** 30), 0xA5, dtype=torch.uint8, device="cuda:0")
    scales = torch.full((1, 2 ** 26), 0xA5, dtype=torch.uint8, device="cuda:0")
    vals = torch.full((2 ** 31,), -7.0, dtype=torch.bfloat16, device="cuda:0")
    q.qtip_mx_quantize(x, SRC["bf16"], 1, cols, cols, RULE["nearest"], codes, scales, vals)
    torch.cuda.synchronize()
    whole = cols // part                                   # repetitions before the last, shorter one
    for got, want in zip((codes[0], scales[0], vals), ref):
        rows = got.view(-1, want.shape[1])
        want = torch.from_numpy(want).to(got.dtype).cuda()
        assert all(bool((piece == want).all()) for piece in rows[:whole].split(2 ** 13))
    rest = cols - whole * part
    tail = mx.quantise(base[:, :rest].double().numpy(), "nearest")
    assert np.array_equal(codes[0, whole * part // 2:].cpu().numpy()[:tail[0].shape[1]], tail[0][0])
    assert np.array_equal(scales[0, whole * part // 32:].cpu().numpy()[:tail[1].shape[1]], tail[1][0])
    assert np.array_equal(vals[whole * part:cols].double().cpu().numpy(), tail[2][0])
    assert bool((vals[cols:] == -7.0).all())


@pytest.mark.parametrize("rule", ["floor", "nearest"])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_quantise_borders_and_extremes(kind, rule):
    import torch
    say(f"quantise borders {kind} {rule}")
    t = dtype_of(kind)
    # every border of the codes and its two neighbours, in blocks whose amax fixes the scale to 2^e
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.99])
    rows = []
    for e in (-12, -3, 0, 5):
        base = (border * 2.0 ** e).to(t)
        up, down = (torch.nextafter(base.float(), torch.tensor(s)).to(t) for s in (np.inf, -np.inf))
        bits = torch.int16 if t != torch.float32 else torch.int32
        up, down = (base.view(bits) + 1).view(t), (base.view(bits) - 1).view(t)
        row = torch.cat([base, -up, down, torch.full((5,), 4.0 * 2.0 ** e).to(t)])
        rows += [row, -row]
    check_quantise(torch.stack(rows).cuda(), kind, rule)
    # powers of two over the type's whole range, subnormal ones among them, zeros, infinities, NaN
    info = torch.finfo(t)
    low = int(np.log2(info.smallest_normal)) - (10 if t == torch.float16 else 7 if t == torch.bfloat16 else 23)
    high = int(np.floor(np.log2(info.max)))
    x = torch.zeros(high - low + 6, 32)
    for i, e in enumerate(range(low, high + 1)):
        x[i, 3], x[i, 7], x[i, 30] = 2.0 ** e, -(2.0 ** max(e - 2, low)), 2.0 ** max(e - 4, low)
    x = x.to(t)
    n = high - low + 1
    x[n] = info.max
    x[n + 1, 9] = float("inf")
    x[n + 2, 31] = float("nan")
    x[n + 3, 0], x[n + 3, 1] = -0.0, info.max
    check_quantise(x.cuda(), kind, rule)


def product(a, w, kind):
    import torch
    dev = [torch.from_numpy(t).cuda() for t in (*a, *w)]
    m, n, k = a[0].shape[0], w[0].shape[0], a[0].shape[1] * 2
    out = torch.full((m, n), -7.0, dtype=dtype_of(kind), device="cuda:0")
    q.qtip_mx_matmul(dev[0], dev[1], m, dev[2], dev[3], n, k, out, OUT[kind])
    torch.cuda.synchronize()
    return out.cpu().double().numpy()


def check_product(a, w, kind):
    av, wv = values(*a), values(*w)
    ref = av @ wv.T
    got = product(a, w, kind)
    err = np.abs(got - ref)
    lim = rounded(sum_bound(av, wv), ref, kind)
    assert np.all(err <= lim), (float((err / lim).max()), np.argwhere(err > lim)[:4].tolist())


SIZES = [(1, 1, 32), (1, 16, 64), (1, 4096, 512), (2, 17, 96), (3, 100, 544), (15, 33, 1056), (16, 16, 2048),
         (17, 64, 512), (33, 48, 4096), (64, 130, 640), (65, 128, 128), (100, 257, 416), (128, 256, 256),
         (129, 72, 992), (255, 300, 1024), (256, 256, 4096), (300, 513, 160), (513, 1040, 2080), (1, 24, 8192),
         (40, 50, 96), (20, 70, 32), (700, 300, 128), (520, 264, 1184)]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_matches_float64(m, n, k, kind):
    say(f"product {m}x{n}x{k} {kind}")
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    check_product(packed(rng, m, k), packed(rng, n, k), kind)


# every tile of the dense product: rows and columns past the tiles' ends, runs of inputs not full
TILES = [(20, 8200, 96), (130, 4100, 1120), (280, 2056, 96), (290, 2050, 4160), (260, 4104, 2080), (300, 3300, 160),
         (1000, 2056, 160), (1001, 2063, 288), (1030, 3200, 96), (1100, 3207, 544), (4000, 4100, 64),
         (3850, 4351, 352)]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", TILES)
def test_large_product_matches_float64(m, n, k, kind):
    say(f"product {m}x{n}x{k} {kind}")
    rng = np.random.default_rng(m * 5 + n + k)
    check_product(packed(rng, m, k), packed(rng, n, k), kind)


def test_product_one_block_at_a_time():
    # one nonzero block per row pair at a time shows any mismatch of codes, scales and lanes exactly
    say("product block by block")
    rng = np.random.default_rng(4)
    k = 1024
    for b in range(k // 32):
        a, w = packed(rng, 16, k), packed(rng, 16, k)
        keep = np.zeros(k // 2, bool)
        keep[16 * b:16 * b + 16] = True
        a[0][:, ~keep] = 0
        got = product(a, w, "fp32")
        assert np.array_equal(got, values(*a) @ values(*w).T), b   # 32 products: exact in fp32


@pytest.mark.parametrize("m,n,k", [(1, 200, 160), (40, 300, 544), (300, 2050, 96), (1000, 2056, 160),
                                   (1030, 3200, 96), (4000, 4100, 64)])
def test_a_nan_block_reaches_its_own_outputs_only(m, n, k):
    say(f"product {m}x{n}x{k} with NaN blocks")
    rng = np.random.default_rng(m + n)
    a, w = packed(rng, m, k), packed(rng, n, k)
    before = product(a, w, "fp32")
    a[1][m - 1, -1] = 255                 # the last block of the last row
    w[1][n - 1, -1] = w[1][n // 2, 0] = 255
    after = product(a, w, "fp32")
    hit = np.zeros((m, n), bool)
    hit[m - 1] = hit[:, n - 1] = hit[:, n // 2] = True
    assert np.all(np.isnan(after[hit]))
    assert np.array_equal(after[~hit], before[~hit])


def test_product_scale_extremes_and_nan_blocks():
    say("product scale extremes")
    rng = np.random.default_rng(6)
    a, w = packed(rng, 20, 256), packed(rng, 40, 256)
    a[1][:] = rng.integers(0, 20, a[1].shape)                       # 2^-127 and above
    w[1][:] = rng.integers(200, 230, w[1].shape)
    check_product(a, w, "fp32")
    a, w = packed(rng, 20, 256), packed(rng, 40, 256)
    a[1][3, 2] = 255
    w[1][7, 5] = 255
    w[1][39, 0] = 255
    a[0][3, 32:48] = 0                                               # a NaN block with zero codes
    got = product(a, w, "fp32")
    bad = np.zeros((20, 40), bool)
    bad[3], bad[:, 7], bad[:, 39] = True, True, True
    assert np.array_equal(np.isnan(got), bad)
    ref = np.where(bad, 0.0, np.nan_to_num(values(*a)) @ np.nan_to_num(values(*w)).T)
    lim = sum_bound(np.nan_to_num(values(*a)), np.nan_to_num(values(*w)))
    assert np.all(np.abs(np.where(bad, 0.0, got) - ref) <= lim + 1e-38)


class Experts:
    """A plan, random MXFP4 weights (numpy and device) and a routed batch."""

    def __init__(self, seed, n, E, k, H, I, skew=False, holes=0.0, max_tokens=None):
        import torch
        rng = np.random.default_rng(seed)
        self.n, self.E, self.k, self.H, self.I = n, E, k, H, I
        self.plan = q.qtip_moe_plan(q.make_desc(E, k, H, I, max_tokens or n), 0)
        self.w = {name: packed(rng, E * rows, cols, 112, 120)
                  for name, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I))}
        self.dev = {name: [torch.from_numpy(t).cuda() for t in v] for name, v in self.w.items()}
        self.weights = q.make_mx_weights(*self.dev["gate"], *self.dev["up"], *self.dev["down"])
        self.idx, self.counts, self.offsets, self.order = bins_of(rng, n, E, k, skew, holes)
        self.x = packed(rng, n, H, 122, 127)
        self.h = packed(rng, n * k, I, 122, 127)

    def run(self, part, kind, offsets=None, order=None):
        import torch
        act, width = (self.x, self.I) if part == "gate_up" else (self.h, self.H)
        full = np.full(self.n * self.k, -9, np.int32)
        full[:len(self.order)] = self.order
        dev = [torch.from_numpy(np.ascontiguousarray(t)).cuda()
               for t in (*act, self.offsets if offsets is None else offsets, full if order is None else order)]
        out = torch.full((self.n * self.k, width), -7.0, dtype=dtype_of(kind), device="cuda:0")
        q.qtip_mx_expert_matmul(self.plan, q.QTIP_MX_PASS_GATE_UP if part == "gate_up" else q.QTIP_MX_PASS_DOWN,
                                self.weights, *dev, self.n, out, OUT[kind])
        torch.cuda.synchronize()
        return out.cpu().double().numpy()

    def check(self, part, kind):
        got = self.run(part, kind)
        flat = self.idx.reshape(-1)
        for e in range(self.E):
            pairs = np.flatnonzero(flat == e)
            if not len(pairs):
                continue
            if part == "gate_up":
                a = values(*self.x)[pairs // self.k]
                g, u = (values(*(t[e * self.I:(e + 1) * self.I] for t in self.w[name])) for name in ("gate", "up"))
                gr, ur = a @ g.T, a @ u.T
                ref = mx.silu(gr) * ur
                # silu itself: exp, add and divide in fp32, a few steps of 2^-24 relative
                lim = mx.swiglu_bound(gr, ur, sum_bound(a, g), sum_bound(a, u)) + 8 * 2.0 ** -24 * np.abs(ref)
            else:
                a = values(*self.h)[pairs]
                d = values(*(t[e * self.H:(e + 1) * self.H] for t in self.w["down"]))
                ref, lim = a @ d.T, sum_bound(a, d)
            lim = rounded(lim, ref, kind)
            err = np.abs(got[pairs] - ref)
            assert np.all(err <= lim), (e, float((err / lim).max()))
        assert np.all(got[np.flatnonzero(flat < 0)] == -7.0)       # pairs in no bin: left as they were

    def close(self):
        q.qtip_moe_plan_destroy(self.plan)


SHAPES = [
    # n, E, k, H, I, skew, holes
    (1, 8, 2, 256, 128, False, 0.0),
    (1, 1, 1, 128, 128, False, 0.0),
    (3, 64, 6, 512, 384, False, 0.0),
    (16, 4, 4, 640, 256, False, 0.0),
    (40, 16, 3, 1152, 128, True, 0.0),
    (70, 5, 2, 384, 640, False, 0.3),
    (200, 8, 2, 256, 256, True, 0.1),
    (17, 300, 4, 128, 256, False, 0.0),
    (600, 3, 2, 512, 256, True, 0.0),
    (260, 2, 2, 2048, 128, False, 0.0),
    (1500, 4, 1, 256, 512, True, 0.05),
]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("part", ["gate_up", "down"])
@pytest.mark.parametrize("n,E,k,H,I,skew,holes", SHAPES)
def test_expert_pass_matches_float64(n, E, k, H, I, skew, holes, part, kind):
    say(f"experts {part} n={n} E={E} k={k} H={H} I={I} skew={skew} holes={holes} {kind}")
    ex = Experts(n * 31 + E, n, E, k, H, I, skew, holes)
    ex.check(part, kind)
    ex.close()


def test_expert_pass_with_no_pair_at_all():
    say("experts without a pair")
    ex = Experts(1, 9, 4, 2, 128, 128, holes=1.0)
    assert np.all(ex.run("gate_up", "bf16") == -7.0)
    assert np.all(ex.run("down", "fp32") == -7.0)
    ex.close()


def test_expert_pass_holds_bad_bins_to_its_bounds():
    # the kernels' own checks: offsets outside [0, n k] are held to it, pair ids outside skipped
    say("experts bad bins")
    ex = Experts(2, 30, 4, 2, 256, 128)
    good = ex.run("down", "fp32")
    order = np.concatenate([ex.order]).astype(np.int32)
    order[[3, 20]] = [60, -2 ** 31]
    got = ex.run("down", "fp32", order=order)
    lost = ex.order[[3, 20]]
    keep = np.setdiff1d(np.arange(60), lost)
    assert np.array_equal(got[keep], good[keep]) and np.all(got[lost] == -7.0)
    offsets = ex.offsets.copy()
    offsets[-1] = 2 ** 31 - 1
    assert np.array_equal(ex.run("down", "fp32", offsets=offsets), good)
    offsets[0] = -5
    assert np.array_equal(ex.run("down", "fp32", offsets=offsets), good)
    ex.close()


def test_results_do_not_depend_on_the_run():
    say("experts same bits twice")
    ex = Experts(7, 333, 6, 3, 512, 256, skew=True)
    for part in ("gate_up", "down"):
        assert np.array_equal(ex.run(part, "fp32"), ex.run(part, "fp32"))
    ex.close()


def test_binding_refuses_tensors_that_do_not_hold_the_call():
    import torch
    say("mx binding refusals")
    dev = dict(device="cuda:0")
    x, c, s = torch.zeros(4, 64, **dev), torch.zeros(4, 32, dtype=torch.uint8, **dev), torch.zeros(
        4, 2, dtype=torch.uint8, **dev)
    call = lambda src=x, kind="fp32", rows=4, cols=64, stride=64, codes=c, scales=s, values=None: q.qtip_mx_quantize(
        src, SRC[kind], rows, cols, stride, 0, codes, scales, values)
    call()
    for bad in (dict(src=x.cpu()), dict(kind="bf16"), dict(rows=5), dict(stride=65), dict(codes=c[:3]),
                dict(scales=s[:, :1]), dict(codes=c.cpu()), dict(values=x[:, :32]), dict(values=x.half())):
        with pytest.raises(q.QtipError):
            call(**bad)
    y = torch.zeros(4, 4, **dev)
    mm = lambda a=c, sa=s, m=4, w=c, sw=s, n=4, k=64, out=y: q.qtip_mx_matmul(a, sa, m, w, sw, n, k, out, OUT["fp32"])
    mm()
    for bad in (dict(a=c.cpu()), dict(m=5), dict(n=5), dict(k=96), dict(out=y.half()), dict(out=y.t()[:2]),
                dict(sw=s.t().contiguous().t())):
        with pytest.raises(q.QtipError):
            mm(**bad)
    torch.cuda.synchronize()
