"""The e4m3 path as it is used: norm, router, gate and experts one after the other, alone, captured, on other streams."""
import numpy as np
import pytest

import trellis_quantized_moe_expert_amd as q
from f8_util import HALF, TYPE, packed, same, sum_bound, within
from gpu_util import say
from oracle import f8, mx

pytestmark = pytest.mark.gpu

EPS = 1e-6


def make(*shape, dtype="float32", fill=None):
    import torch
    t = torch.empty(shape, dtype=getattr(torch, dtype), device="cuda:0")
    return t.fill_(float("nan") if fill is None and t.is_floating_point() else 0xA5 if fill is None else fill)


class Block:
    """The feed-forward half of a model's layer: residual sum and norm into e4m3, router product, gate, experts."""

    def __init__(self, seed, n, E, k, H, I, out_dtype="bf16", gated=True, max_tokens=None):
        import torch
        rng = np.random.default_rng(seed)
        self.n, self.E, self.k, self.H, self.I, self.out_dtype = n, E, k, H, I, out_dtype
        kind = q.QTIP_OUT_BF16 if out_dtype == "bf16" else q.QTIP_OUT_F32
        self.plan = q.qtip_moe_plan(q.make_desc(E, k, H, I, max_tokens or n, out_dtype=kind), 0)
        self.w = {m: packed(rng, E * rows, cols, 128, -16, -12)
                  for m, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I))}
        self.dev = {m: [torch.from_numpy(t).cuda() for t in v] for m, v in self.w.items()}
        self.weights = q.make_f8_weights(*self.dev["gate"], *self.dev["up"], *self.dev["down"])
        f32 = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()
        self.norm_w = (1 + 0.1 * f32(H)).bfloat16()
        self.router = (f32(E, H) / np.sqrt(H)).bfloat16()
        self.gate = q.make_gate(q.QTIP_GATE_SIGMOID, bias=0.05 * f32(E), scale=2.5) if gated else None
        self.ws = make(q.qtip_f8_moe_workspace_bytes(self.plan), dtype="uint8", fill=255)
        self.router_ws = make(q.qtip_moe_plan_info(self.plan)["workspace_bytes"], dtype="uint8", fill=255)
        self.x, self.res = self.tokens(rng)
        self.bufs = self.buffers()

    def tokens(self, rng):
        import torch
        f32 = lambda: torch.from_numpy(rng.standard_normal((self.n, self.H)).astype(np.float32)).cuda()
        return f32().bfloat16(), (3 * f32()).bfloat16()

    def buffers(self):
        n, E, H = self.n, self.E, self.H
        return dict(codes=make(n, H, dtype="uint8"), scales=make(n, H // 128), sums=make(n, H, dtype="bfloat16"),
                    values=make(n, H, dtype="bfloat16"), logits=make(n, E),
                    out=make(n, H, dtype="bfloat16" if self.out_dtype == "bf16" else "float32"))

    def run(self, b=None, x=None, res=None, ws=None):
        b = b or self.bufs
        x, res, ws = (self.x if x is None else x), (self.res if res is None else res), (self.ws if ws is None else ws)
        n, H = self.n, self.H
        q.qtip_f8_rms_norm(x, TYPE["bf16"], n, H, H, res, H, b["sums"], self.norm_w, TYPE["bf16"], EPS,
                           q.QTIP_F8_SCALE_AMAX, b["codes"], b["scales"], b["values"])
        q.qtip_moe_router_logits(self.plan, b["values"], self.router, n, b["logits"], self.router_ws,
                                 self.router_ws.numel())
        self.layer(b, ws)
        return b

    def layer(self, b, ws=None, out=None):
        ws = self.ws if ws is None else ws
        q.qtip_f8_moe_forward(self.plan, self.weights, self.gate, b["codes"], b["scales"], b["logits"], self.n,
                              b["out"] if out is None else out, ws, ws.numel())

    def steps(self, b):
        """(expert ids, weights, h codes, h scales, y) of the layer's own steps."""
        import torch
        n, E, k, H, I = self.n, self.E, self.k, self.H, self.I
        i32 = lambda *s: make(*s, dtype="int32", fill=0)
        idx, w, counts, offs, order = i32(n, k), make(n, k), i32(E), i32(E + 1), i32(n * k)
        if self.gate is None:
            q.qtip_moe_route(self.plan, b["logits"], n, idx, w, counts, offs, order, i32(n * k, 3), i32(1))
        else:
            gws = make(q.qtip_moe_gate_workspace_bytes(self.plan), dtype="uint8")
            q.qtip_moe_gate_route(self.plan, self.gate, b["logits"], n, idx, w, counts, offs, order, None, None, gws,
                                  gws.numel())
        hc, hs, y = make(n * k, I, dtype="uint8"), make(n * k, I // 128), make(n * k, H, fill=0.0)
        q.qtip_f8_expert_matmul(self.plan, q.QTIP_F8_PASS_GATE_UP, self.weights, b["codes"], b["scales"], offs, order, n,
                                hc, q.QTIP_OUT_E4M3, hs)
        q.qtip_f8_expert_matmul(self.plan, q.QTIP_F8_PASS_DOWN, self.weights, hc, hs, offs, order, n, y, q.QTIP_OUT_F32)
        torch.cuda.synchronize()
        return (idx.cpu().numpy(), w.double().cpu().numpy(), hc.cpu().numpy(), hs.cpu().numpy(),
                y.double().cpu().numpy().reshape(n, k, H))

    def matrix(self, name, e):
        rows = self.H if name == "down" else self.I
        codes, scales = self.w[name]
        return f8.decode(codes[e * rows:(e + 1) * rows], scales[e * rows // 128:(e + 1) * rows // 128], 128)

    def close(self):
        q.qtip_moe_plan_destroy(self.plan)


def numbers(t):
    return t.double().cpu().numpy()


def bits(b):
    import torch
    torch.cuda.synchronize()
    return {name: t.cpu().contiguous().view(torch.uint8).numpy().copy() for name, t in b.items()}


def equal(a, b):
    for name in a:
        assert bool(np.array_equal(a[name], b[name])), name


def combined(parts):
    """The weighted sum over a token's pairs in float64, and a bound of the combine's fp32 error."""
    return parts.sum(1), parts.shape[1] * 2.0 ** -24 * np.abs(parts).sum(1)


SHAPES = [(1, 8, 2, 256, 128), (16, 8, 3, 512, 384), (17, 64, 6, 384, 256), (150, 8, 2, 256, 640), (700, 4, 2, 384, 128)]


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n,E,k,H,I", SHAPES)
def test_layer_is_its_steps(n, E, k, H, I, gated, out_dtype):
    say(f"e4m3 layer n={n} E={E} k={k} H={H} I={I} gated={gated} {out_dtype}")
    blk = Block(n + E, n, E, k, H, I, out_dtype, gated)
    b = blk.run()
    idx, w, _, _, y = blk.steps(b)
    assert idx.min() >= 0
    ref, bound = combined(w[:, :, None] * y)
    within(numbers(b["out"]), ref, bound + HALF[out_dtype] * (np.abs(ref) + bound))
    # a part of the plan's tokens, and a workspace that holds anything
    blk.close()


@pytest.mark.parametrize("n,E,k,H,I", [(3, 8, 2, 256, 128), (40, 8, 2, 512, 256)])
def test_block_matches_float64(n, E, k, H, I):
    # each stage from the last one's device results, so that a rounding to 8 bits is not blamed on the next stage
    say(f"e4m3 block n={n}")
    blk = Block(n, n, E, k, H, I, "fp32")
    b = blk.run()
    h = numbers(blk.x) + numbers(blk.res)
    sums = numbers(b["sums"])
    within(sums, h, HALF["bf16"] * np.abs(h))
    y = f8.rms_norm(sums, numbers(blk.norm_w), EPS)
    codes, scales = b["codes"].cpu().numpy(), b["scales"].cpu().numpy()
    x = f8.decode(codes, scales)
    s = scales.astype(np.float64).repeat(128, axis=1)
    within(x, y, np.maximum(2.0 ** -4 * np.abs(y), s * 2.0 ** -10) * (1 + 1e-5))     # half a step of e4m3
    values = numbers(b["values"])
    within(values, y, (HALF["bf16"] + 1e-5) * np.abs(y))
    idx, w, hc, hs, _ = blk.steps(b)
    hv = f8.decode(hc, hs).reshape(n, k, I)
    ref, lim = np.zeros((n, H)), np.zeros((n, H))
    for t in range(n):
        for j in range(k):
            g, u, d = (blk.matrix(name, idx[t, j]) for name in ("gate", "up", "down"))
            row = x[t:t + 1]
            gr, ur = row @ g.T, row @ u.T
            want = mx.silu(gr) * ur
            off = mx.swiglu_bound(gr, ur, sum_bound(row, g, H // 128), sum_bound(row, u, H // 128)) + 2.0 ** -21 * np.abs(want)
            got = hv[t, j:j + 1]
            step = np.maximum(2.0 ** -4 * (np.abs(want) + off), hs.reshape(n, k, -1)[t, j].repeat(128) * 2.0 ** -10)
            within(got, want, off + step)
            ref[t] += w[t, j] * (got @ d.T)[0]
            lim[t] += abs(w[t, j]) * (sum_bound(got, d, I // 128)[0] + k * 2.0 ** -23 * np.abs(got @ d.T)[0])
    within(numbers(b["out"]), ref, lim + HALF["fp32"] * np.abs(ref))
    blk.close()


def test_tokens_without_an_expert_get_zeros():
    say("e4m3 layer with experts taken out")
    import torch
    blk = Block(5, 20, 8, 2, 256, 128, "fp32")
    blk.gate = q.make_gate(q.QTIP_GATE_SIGMOID, bias=torch.tensor([0.0] + [-np.inf] * 7, device="cuda:0"))
    b = blk.run()
    b["logits"][3] = -np.inf
    blk.layer(b)
    idx, w, _, _, y = blk.steps(b)
    assert np.all(idx[:, 1] == -1) and np.all(idx[3] == -1)
    out = numbers(b["out"])
    assert not out[3].any()
    keep = np.arange(20) != 3
    within(out[keep], (w[:, :1] * y[:, 0])[keep], 2.0 ** -23 * np.abs(w[:, :1] * y[:, 0])[keep])
    blk.close()


def test_fewer_tokens_than_the_plan_holds():
    # rows behind the last token stay as they were; nothing of an earlier call in the workspace is read
    say("e4m3 layer of fewer tokens")
    import torch
    blk = Block(6, 9, 8, 2, 256, 128, max_tokens=300)
    want = bits(blk.run(blk.buffers()))
    wide = make(12, 256, dtype="bfloat16", fill=-7.0)
    codes = make(12, 256, dtype="uint8")
    blk.ws.fill_(17)
    b = dict(blk.buffers(), out=wide, codes=codes)
    blk.run(b)
    torch.cuda.synchronize()
    assert np.array_equal(wide[:9].contiguous().view(torch.uint8).cpu().numpy(), want["out"])
    assert bool((wide[9:] == -7.0).all()) and bool((codes[9:] == 0xA5).all())
    blk.close()


@pytest.mark.parametrize("n,E,k,H,I", [(1, 8, 2, 256, 128), (40, 8, 2, 512, 256), (300, 4, 2, 256, 256)])
def test_two_captured_graphs_replay_the_block(n, E, k, H, I):
    # two graphs over one plan and the same weights, a workspace each, replayed in turn with eager work between
    import torch
    say(f"e4m3 graphs n={n}")
    blk = Block(n + 9, n, E, k, H, I)
    other = blk.tokens(np.random.default_rng(77))
    want = bits(blk.run(blk.buffers()))
    want_other = bits(blk.run(blk.buffers(), *other))
    graphs = []
    for _ in range(2):
        buf, x, res, ws = blk.buffers(), blk.x.clone(), blk.res.clone(), torch.zeros_like(blk.ws)
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                blk.run(buf, x, res, ws)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        graphs.append((g, buf, x, res, ws))
    eager = blk.buffers()
    for rep in range(3):
        for g, buf, x, res, _ in graphs:
            for t in buf.values():
                t.fill_(0 if not t.is_floating_point() else float("nan"))
            blk.run(eager, *other)
            torch.cuda.synchronize()
            g.replay()
            equal(bits(buf), want)
            equal(bits(eager), want_other)
    g, buf, x, res, _ = graphs[1]
    x.copy_(other[0])
    res.copy_(other[1])
    g.replay()
    equal(bits(buf), want_other)
    g, buf, x, res, _ = graphs[0]
    g.replay()
    equal(bits(buf), want)
    blk.close()


def test_two_streams_at_once():
    import torch
    say("e4m3 on two streams")
    blks = [Block(3, 200, 8, 2, 512, 256), Block(4, 30, 8, 2, 512, 256)]
    want = [bits(blk.run(blk.buffers())) for blk in blks]
    streams = [torch.cuda.Stream() for _ in blks]
    torch.cuda.synchronize()
    got = [blk.buffers() for blk in blks]
    torch.cuda.synchronize()
    for _ in range(5):
        for blk, s, b in zip(blks, streams, got):
            with torch.cuda.stream(s):       # calls take the current stream
                blk.run(b)
    for b, ref, blk in zip(got, want, blks):
        equal(bits(b), ref)
        blk.close()


def test_dense_chain_quantise_then_product():
    # a linear layer as it is used: weights brought to e4m3 once, activations on the way
    import torch
    say("e4m3 linear")
    g = torch.Generator().manual_seed(5)
    m, n, k = 70, 200, 1000
    x, w = torch.randn(m, k, generator=g).bfloat16().cuda(), (torch.randn(n, k, generator=g) / k ** 0.5).cuda()
    kp = 1008
    ac, asc, wc, wsc = make(m, kp, dtype="uint8"), make(m, 8), make(n, kp, dtype="uint8"), make(2, 8)
    q.qtip_f8_quantize(w, TYPE["fp32"], n, k, k, 128, q.QTIP_F8_SCALE_POW2, wc, wsc)
    q.qtip_f8_quantize(x, TYPE["bf16"], m, k, k, 1, q.QTIP_F8_SCALE_AMAX, ac, asc)
    y = make(m, n)
    q.qtip_f8_matmul(ac, asc, m, wc, wsc, n, kp, y, q.QTIP_OUT_F32)
    torch.cuda.synchronize()
    a = f8.quantise(numbers(x), "amax")
    b = f8.quantise(numbers(w), "pow2", 128)
    same((ac.cpu().numpy(), asc.cpu().numpy()), a)
    same((wc.cpu().numpy(), wsc.cpu().numpy()), b)
    av, bv = f8.decode(*a), f8.decode(*b, 128)
    within(numbers(y), av @ bv.T, sum_bound(av, bv, 8) + HALF["fp32"] * np.abs(av @ bv.T))


@pytest.mark.parametrize("m,n,k,kind", [(600_000, 16, 4096, "bf16"), (3, 600_000, 4096, "fp32"), (40, 1_100_000, 2048, "bf16"),
                                        (1_100_000, 130, 2048, "fp32"), (4200, 4112, 8336, "bf16"),
                                        (4200, 4112, 8336, "fp32")])
def test_products_of_large_matrices(m, n, k, kind):
    # rows repeat with a period, so that few of them have to be computed in float64; the last ones are looked at
    import torch
    say(f"e4m3 product {m}x{n}x{k}")
    rng = np.random.default_rng(8)
    rows_a, rows_w = min(m, 96), min(n, 128)
    a, w = packed(rng, rows_a, k), packed(rng, rows_w, k, 128)
    tile = lambda t, count: torch.from_numpy(t).cuda().repeat(-(-count // t.shape[0]), 1)[:count].contiguous()
    w_scales = tile(w[1], -(-n // 128))
    y = make(m, n, dtype="bfloat16" if kind == "bf16" else "float32")
    q.qtip_f8_matmul(tile(a[0], m), tile(a[1], m), m, tile(w[0], n), w_scales, n, k, y,
                     q.QTIP_OUT_BF16 if kind == "bf16" else q.QTIP_OUT_F32)
    torch.cuda.synchronize()
    from f8_util import eight_bound, rounded
    av, wv = f8.decode(*a), f8.decode(*w, 128)
    ref = av @ wv.T
    lim = rounded(sum_bound(av, wv, -(-k // 128)) + (eight_bound(av, wv) if kind == "bf16" else 0.0), ref, kind)
    for r in (0, m // 2, m - 1):
        for c in (0, n // 2, n - 1):
            got = float(y[r, c])
            i, j = r % rows_a, c % rows_w
            assert abs(got - ref[i, j]) <= lim[i, j], (r, c, got, ref[i, j])
    flat = y if m < n else y.t()
    period = rows_w if m < n else rows_a
    first, last = flat[:, :period], flat[:, flat.shape[1] - flat.shape[1] % period - period:][:, :period]
    assert torch.equal(first, last)
