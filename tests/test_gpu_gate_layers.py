"""The operators as a layer runs them: the trellis layer behind a gate against the oracle, and the
MXFP4 layer against its steps taken one by one through their own entry points."""
import numpy as np
import pytest

import moe_inputs
import parity
import trellis_quantized_moe_expert_amd as q
from gpu_util import Layer, say
from moe_inputs.device import tokens_to_device
from mx_util import packed
from oracle import gate as oracle
from oracle import moe

pytestmark = pytest.mark.gpu

GATE = dict(score="sigmoid", num_groups=4, top_groups=2, group_top=2, scale=2.5)
SCORES = {"softmax": q.QTIP_GATE_SOFTMAX, "sigmoid": q.QTIP_GATE_SIGMOID}


def make_gate(bias, score, **kw):
    return q.make_gate(score=SCORES[score], bias=bias, **kw)


def masked_logits(logits):
    out = logits.copy()
    out[1] = -np.inf                      # a token without any expert
    out[2, 1:] = -np.inf                  # a token with one
    return out


@pytest.mark.parametrize("rung", ["bitshift", "lut"])
@pytest.mark.parametrize("n,arm", [(3, q.QTIP_ARM_AUTO), (16, q.QTIP_ARM_GEMV), (50, q.QTIP_ARM_AUTO),
                                   (50, q.QTIP_ARM_DEQUANT)])
def test_gated_trellis_layer_matches_the_oracle(n, arm, rung):
    import torch
    shape = moe_inputs.MoEShape(8, 3, 256, 128, n, rung=rung)
    inp = moe_inputs.make_inputs(shape, seed=4)
    inp.logits[:] = masked_logits(inp.logits)
    rng = np.random.default_rng(n)
    bias = (0.1 * rng.standard_normal(8)).astype(np.float32)
    say(f"gated trellis layer n={n} arm={arm} {rung}")
    layer = Layer(inp, arm=arm)
    t = tokens_to_device(inp)
    b = torch.from_numpy(bias).cuda()
    out = torch.full((n, 256), float("nan"), dtype=torch.float32, device="cuda:0")
    layer.ws.fill_(255)                   # NaN wherever a left-out pair's row would be read
    q.qtip_moe_forward_gated(layer.plan, layer.w, make_gate(b, **GATE), t.x, t.logits, n, out, layer.ws,
                             layer.ws.numel())
    torch.cuda.synchronize()
    got = out.cpu().numpy()
    layer.close()
    idx, w = oracle.route(inp.logits, bias, 3, **GATE)
    _, offsets, order = oracle.bins(idx, 8)
    y = {p: np.zeros(256) for p in range(n * 3)}
    for e in range(8):
        pids = order[offsets[e]:offsets[e + 1]]
        if len(pids):
            y.update(zip(pids.tolist(), moe.expert_pairs(inp, e, pids)[0]))
    ok, st = parity.check_f32(got, moe.combine(y, w, range(n), 3, 256))
    assert ok, st
    assert np.all(got[1] == 0)


class MxLayer:
    def __init__(self, seed, n, E, k, H, I, out_dtype, max_tokens=None):
        import torch
        rng = np.random.default_rng(seed)
        self.n, self.E, self.k, self.H, self.I = n, E, k, H, I
        self.bf16 = out_dtype == "bf16"
        self.plan = q.qtip_moe_plan(q.make_desc(E, k, H, I, max_tokens or n, out_dtype=q.QTIP_OUT_BF16 if self.bf16
                                                else q.QTIP_OUT_F32), 0)
        dev = [torch.from_numpy(t).cuda() for rows, cols in ((I, H), (I, H), (H, I))
               for t in packed(rng, E * rows, cols, 114, 122)]
        self.weights = q.make_mx_weights(*dev)
        self.ws = torch.full((q.qtip_mx_moe_workspace_bytes(self.plan),), 255, dtype=torch.uint8, device="cuda:0")

    def out(self):
        import torch
        return torch.full((self.n, self.H), float("nan"), dtype=torch.bfloat16 if self.bf16 else torch.float32,
                          device="cuda:0")

    def forward(self, gate, x, logits, out):
        q.qtip_mx_moe_forward(self.plan, self.weights, gate, x, logits, self.n, out, self.ws, self.ws.numel())

    def steps(self, gate, x, logits):
        """The layer's output in float64 from its single steps, and a bound of the combine's error."""
        import torch
        n, E, k, H, I = self.n, self.E, self.k, self.H, self.I
        mk = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda:0")
        idx, w, counts, offs, order = mk(n, k), mk(n, k, dt=torch.float32), mk(E), mk(E + 1), mk(n * k)
        tiles, nt = mk(n * k, 3), mk(1)
        if gate is None:
            q.qtip_moe_route(self.plan, logits, n, idx, w, counts, offs, order, tiles, nt)
        else:
            ws = mk(q.qtip_moe_gate_workspace_bytes(self.plan), dt=torch.uint8)
            q.qtip_moe_gate_route(self.plan, gate, logits, n, idx, w, counts, offs, order, None, None, ws, ws.numel())

        def quantise(src, rows, cols):
            c, s = mk(rows, cols // 2, dt=torch.uint8), mk(rows, cols // 32, dt=torch.uint8)
            q.qtip_mx_quantize(src, q.QTIP_MX_SRC_BF16, rows, cols, cols, q.QTIP_MX_SCALE_NEAREST, c, s)
            return c, s
        h, y = mk(n * k, I, dt=torch.bfloat16), mk(n * k, H, dt=torch.float32)
        q.qtip_mx_expert_matmul(self.plan, q.QTIP_MX_PASS_GATE_UP, self.weights, *quantise(x, n, H), offs, order, n, h,
                                q.QTIP_OUT_BF16)
        q.qtip_mx_expert_matmul(self.plan, q.QTIP_MX_PASS_DOWN, self.weights, *quantise(h, n * k, I), offs, order, n, y,
                                q.QTIP_OUT_F32)
        torch.cuda.synchronize()
        parts = (w.double().unsqueeze(2) * y.double().reshape(n, k, H)).cpu().numpy()
        ref = parts.sum(1)
        bound = k * 2.0 ** -24 * np.abs(parts).sum(1)              # k fused multiply-adds in fp32
        return ref, bound + (2.0 ** -8 if self.bf16 else 2.0 ** -24) * (np.abs(ref) + bound), idx.cpu().numpy()

    def close(self):
        q.qtip_moe_plan_destroy(self.plan)


def tokens(rng, n, H, E):
    import torch
    x = torch.from_numpy(rng.standard_normal((n, H)).astype(np.float32)).cuda().to(torch.bfloat16)
    return x, rng.standard_normal((n, E)).astype(np.float32)


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n,E,k,H,I", [(1, 8, 2, 256, 128), (16, 8, 3, 512, 384), (17, 64, 6, 384, 256),
                                       (150, 8, 2, 256, 640), (700, 4, 2, 384, 128)])
def test_mx_layer_is_its_steps(n, E, k, H, I, gated, out_dtype):
    import torch
    rng = np.random.default_rng(n + E)
    layer = MxLayer(n, n, E, k, H, I, out_dtype)
    x, logits = tokens(rng, n, H, E)
    gate = None
    if gated:
        if n > 2:
            logits = masked_logits(logits)
        gate = make_gate(torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32)).cuda(), **GATE)
    say(f"mx layer n={n} E={E} k={k} H={H} I={I} gated={gated} {out_dtype}")
    lg = torch.from_numpy(logits).cuda()
    out = layer.out()
    layer.forward(gate, x, lg, out)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    ref, lim, idx = layer.steps(gate, x, lg)
    assert np.all(np.abs(got - ref) <= lim)
    if gated and n > 2:
        assert np.all(got[1] == 0) and np.all(idx[1] == -1) and (idx[2] >= 0).sum() <= 1
    assert np.abs(got).max() > 0
    layer.close()


def test_mx_layer_captured_and_beside_another():
    import torch
    rng = np.random.default_rng(5)
    n, E, k, H, I = 130, 16, 4, 512, 256
    a, b = MxLayer(1, n, E, k, H, I, "fp32", max_tokens=200), MxLayer(2, n, E, k, H, I, "bf16")
    gate = make_gate(None, **GATE)
    batches = []
    for _ in range(3):
        x, logits = tokens(rng, n, H, E)
        batches.append((x, torch.from_numpy(masked_logits(logits)).cuda()))
    say("mx layer captured")
    want = []
    for x, lg in batches:
        out = a.out()
        a.forward(gate, x, lg, out)
        torch.cuda.synchronize()
        want.append(out.clone())
    x_buf, lg_buf, out = batches[0][0].clone(), batches[0][1].clone(), a.out()
    out_b = b.out()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a.forward(gate, x_buf, lg_buf, out)
    torch.cuda.synchronize()
    first_b = None
    for i in (1, 2, 0, 2):
        x_buf.copy_(batches[i][0])
        lg_buf.copy_(batches[i][1])
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        b.forward(None, batches[0][0], torch.nan_to_num(batches[0][1], neginf=-9.0), out_b)   # with its own workspace
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        first_b = out_b.clone() if first_b is None else first_b
        assert torch.equal(out_b, first_b)
    a.close()
    b.close()


def gated_layer(shape, seed, arm, logits, bias, gate):
    """A trellis layer behind a gate: (GPU output, the oracle's, the oracle's expert ids)."""
    import torch
    inp = moe_inputs.make_inputs(shape, seed=seed)
    n, E, k, H = shape.n_tokens, shape.num_experts, shape.top_k, shape.hidden
    inp.logits[:] = logits
    layer = Layer(inp, arm=arm)
    t = tokens_to_device(inp)
    out = torch.full((n, H), float("nan"), dtype=torch.float32, device="cuda:0")
    layer.ws.fill_(255)                   # NaN wherever a left-out pair's row would be read
    q.qtip_moe_forward_gated(layer.plan, layer.w, make_gate(torch.from_numpy(bias).cuda(), **gate), t.x, t.logits, n, out,
                             layer.ws, layer.ws.numel())
    torch.cuda.synchronize()
    got = out.cpu().numpy()
    layer.close()
    idx, w = oracle.route(inp.logits, bias, k, **gate)
    _, offsets, order = oracle.bins(idx, E)
    y = {p: np.zeros(H) for p in range(n * k)}
    for e in np.unique(idx[idx >= 0]):
        pids = order[offsets[e]:offsets[e + 1]]
        y.update(zip(pids.tolist(), moe.expert_pairs(inp, e, pids)[0]))
    return got, moe.combine(y, w, range(n), k, H), idx


@pytest.mark.parametrize("rung", ["bitshift", "lut"])
@pytest.mark.parametrize("n,E,k,gate", [
    (1, 8, 3, GATE), (1, 300, 6, dict(GATE, group_top=1)), (1, 320, 10, dict(GATE, num_groups=32, top_groups=5)),
    (2, 130, 9, dict(renormalise=0)), (24, 260, 4, GATE), (40, 96, 12, dict(score="sigmoid"))])
def test_gated_trellis_layer_of_one_token_and_of_many_experts(n, E, k, gate, rung):
    rng = np.random.default_rng(E + k)
    say(f"gated trellis layer n={n} E={E} k={k} {rung}")
    shape = moe_inputs.MoEShape(E, k, 256, 128, n, rung=rung)
    logits = rng.standard_normal((n, E)).astype(np.float32)
    if n == 24:
        logits[5, 3:] = -np.inf           # fewer experts left than choices
    got, want, idx = gated_layer(shape, 6, q.QTIP_ARM_AUTO, logits, (0.1 * rng.standard_normal(E)).astype(np.float32),
                                 dict(dict(score="softmax"), **gate))
    ok, st = parity.check_f32(got, want)
    assert ok, st
    assert (idx >= 0).any() and np.abs(got).max() > 0


@pytest.mark.parametrize("rung", ["bitshift", "lut"])
@pytest.mark.parametrize("n,arm", [(1, q.QTIP_ARM_AUTO), (1, q.QTIP_ARM_GROUPED), (20, q.QTIP_ARM_GEMV),
                                   (20, q.QTIP_ARM_GROUPED), (20, q.QTIP_ARM_DEQUANT), (200, q.QTIP_ARM_GROUPED)])
def test_gated_trellis_layer_without_any_expert(n, arm, rung):
    say(f"gated trellis layer n={n} arm={arm} {rung}, no expert left")
    shape = moe_inputs.MoEShape(8, 3, 256, 128, n, rung=rung)
    logits = np.full((n, 8), -np.inf, np.float32)
    got, _, idx = gated_layer(shape, 7, arm, logits, np.zeros(8, np.float32), GATE)
    assert np.all(idx == -1) and np.all(got == 0)


def test_mx_layer_without_any_expert_and_of_many():
    import torch
    say("mx layer, no expert left; 300 experts, 10 choices")
    rng = np.random.default_rng(9)
    for n in (1, 40):
        layer = MxLayer(3, n, 8, 2, 256, 128, "fp32")
        x, _ = tokens(rng, n, 256, 8)
        out = layer.out()
        layer.forward(make_gate(None, **GATE), x, torch.full((n, 8), -float("inf"), device="cuda:0"), out)
        torch.cuda.synchronize()
        assert bool((out == 0).all())
        layer.close()
        layer = MxLayer(4, n, 300, 10, 128, 128, "fp32")
        x, logits = tokens(rng, n, 128, 300)
        gate, lg, out = make_gate(None, "sigmoid", num_groups=4, top_groups=2), torch.from_numpy(logits).cuda(), layer.out()
        layer.forward(gate, x, lg, out)
        torch.cuda.synchronize()
        ref, lim, idx = layer.steps(gate, x, lg)
        assert np.all(idx >= 0) and np.all(np.abs(out.double().cpu().numpy() - ref) <= lim)
        layer.close()
