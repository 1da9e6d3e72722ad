"""Refusals of the gate's and MXFP4's entry points: every one is decided on the host, before any
device work, so plain integers stand for device addresses here."""
import ctypes
import math

import pytest

import trellis_quantized_moe_expert_amd as q

V4 = dict(num_experts=256, top_k=6, hidden=4096, inter=2048, max_tokens=64)
ARG, CONFIG = q.QTIP_ERR_INVALID_ARG, q.QTIP_ERR_INVALID_CONFIG


@pytest.fixture
def plan():
    p = q.qtip_moe_plan_for_arch(q.make_desc(**V4), "gfx950")
    yield p
    q.qtip_moe_plan_destroy(p)


def gate_call(plan, gate, logits=256, n=4, idx=256, offsets=256, tile_map=256, n_tiles=256, ws=256, size=None):
    size = q.qtip_moe_gate_workspace_bytes(plan) if size is None else size
    return q.raw_status("qtip_moe_gate_route", plan, None if gate is None else ctypes.byref(gate), logits, n, idx, 256,
                        256, offsets, 256, tile_map, n_tiles, ws, size, None)


@pytest.mark.parametrize("bad", [
    dict(score=2), dict(score=-1), dict(num_groups=0), dict(num_groups=7), dict(num_groups=128, top_groups=128),
    dict(num_groups=8, top_groups=0), dict(num_groups=8, top_groups=9), dict(num_groups=64, top_groups=1),
    dict(group_top=0), dict(group_top=3), dict(renormalise=2), dict(scale=math.inf), dict(scale=math.nan),
    dict(bias=258)])
def test_bad_gates_are_refused(plan, bad):
    gate = q.make_gate(**bad)
    assert gate_call(plan, gate) == ARG
    assert "gate" in q.last_error_detail()
    ws = q.qtip_moe_plan_info(plan)["workspace_bytes"]
    w = q.make_weights(*[256] * 7)
    assert q.raw_status("qtip_moe_forward_gated", plan, ctypes.byref(w), ctypes.byref(gate), 256, 256, 4, 256, 256, ws,
                        None) == ARG
    mw = q.make_mx_weights(*[256] * 6)
    assert q.raw_status("qtip_mx_moe_forward", plan, ctypes.byref(mw), ctypes.byref(gate), 256, 256, 4, 256, 256,
                        q.qtip_mx_moe_workspace_bytes(plan), None) == ARG


def test_gate_route_refusals(plan):
    gate = q.make_gate()
    size = q.qtip_moe_gate_workspace_bytes(plan)
    assert size > 0 and q.qtip_moe_gate_workspace_bytes(None) == 0
    assert gate_call(plan, None) == ARG
    assert gate_call(None, gate, size=size) == ARG
    for name in ("logits", "idx", "offsets", "ws"):
        assert gate_call(plan, gate, **{name: None}) == ARG
    assert gate_call(plan, gate, tile_map=None) == ARG
    assert gate_call(plan, gate, n_tiles=None) == ARG
    assert gate_call(plan, gate, size=size - 1) == ARG
    assert gate_call(plan, gate, ws=384) == ARG
    for n in (0, -1, 65):
        assert gate_call(plan, gate, n=n) == CONFIG


def test_gated_forward_refusals(plan):
    ws = q.qtip_moe_plan_info(plan)["workspace_bytes"]
    w, gate = q.make_weights(*[256] * 7), q.make_gate()
    call = lambda g=gate, x=256, lg=256, n=4, out=256, wsp=256, size=ws: q.raw_status(
        "qtip_moe_forward_gated", plan, ctypes.byref(w), None if g is None else ctypes.byref(g), x, lg, n, out, wsp,
        size, None)
    assert call(g=None) == ARG and call(x=None) == ARG and call(lg=None) == ARG and call(out=None) == ARG
    assert call(wsp=None) == ARG and call(size=ws - 1) == ARG and call(wsp=384) == ARG
    assert call(n=0) == CONFIG and call(n=65) == CONFIG


def test_quantize_refusals():
    def call(src=256, kind=q.QTIP_MX_SRC_BF16, rows=4, cols=64, stride=64, rule=q.QTIP_MX_SCALE_FLOOR, codes=256,
             scales=256, values=256):
        return q.raw_status("qtip_mx_quantize", src, kind, rows, cols, stride, rule, codes, scales, values, None)
    assert call(src=None) == ARG and call(codes=None) == ARG and call(scales=None) == ARG
    assert call(kind=3) == ARG and call(kind=-1) == ARG and call(rule=2) == ARG
    assert call(rows=0) == CONFIG and call(cols=0) == CONFIG and call(rows=-1) == CONFIG
    assert call(stride=63) == ARG and call(stride=1 << 40) == ARG
    assert call(src=257) == ARG and call(src=258, kind=q.QTIP_MX_SRC_F32) == ARG
    assert call(codes=264) == ARG and call(values=264) == ARG
    assert call(rows=1 << 30, cols=64) == ARG                   # 2^31 blocks
    assert call(cols=2 ** 31 - 1, rows=64, stride=2 ** 31) == ARG


def test_matmul_refusals():
    def call(a=256, sa=256, m=4, w=256, sw=256, n=32, k=64, out=256, kind=q.QTIP_OUT_F32):
        return q.raw_status("qtip_mx_matmul", a, sa, m, w, sw, n, k, out, kind, None)
    for name in ("a", "sa", "w", "sw", "out"):
        assert call(**{name: None}) == ARG
    assert call(kind=2) == ARG and call(k=48) == ARG
    assert call(m=0) == CONFIG and call(n=0) == CONFIG and call(k=0) == CONFIG and call(m=-4) == CONFIG
    assert call(a=264) == ARG and call(w=264) == ARG and call(out=264) == ARG and call(sa=257) == ARG
    assert call(sw=258) == ARG
    assert call(m=1 << 30, k=128) == ARG and call(n=1 << 30, k=128) == ARG
    assert call(m=1 << 20, n=1 << 20, k=32) == ARG


def test_launches_past_2_32_threads_are_refused():
    # four threads a block of 32 values; 256 threads for 16 weight rows; 512 for 256 x 256 outputs
    quantize = lambda rows, cols: q.raw_status("qtip_mx_quantize", 256, q.QTIP_MX_SRC_BF16, rows, cols, cols,
                                               q.QTIP_MX_SCALE_FLOOR, 256, 256, None, None)
    assert quantize(1 << 30, 32) == ARG and quantize((1 << 30) - 63, 32) == ARG and quantize(1 << 20, 1 << 15) == ARG
    matmul = lambda m, n: q.raw_status("qtip_mx_matmul", 256, 256, m, 256, 256, n, 32, 256, q.QTIP_OUT_F32, None)
    assert matmul(1, 1 << 28) == CONFIG and matmul(16, (1 << 28) - 15) == CONFIG
    assert matmul(1 << 19, (1 << 21) - 256) == CONFIG and "threads" in q.last_error_detail()


@pytest.mark.parametrize("m,n", [(1, 2 ** 31 - 16), (1, 2 ** 31 - 15), (1, 2 ** 31 - 1), (16, 2 ** 31 - 1),
                                 (17, 2 ** 31 - 1), (300, 2 ** 31 - 130), (511, 2 ** 31 - 1), (2 ** 31 - 1, 1),
                                 (2 ** 31 - 1, 16), (2 ** 31 - 255, 300), (2 ** 31 - 257, 511)])
def test_products_of_rows_next_to_2_31_are_refused(m, n):
    # the launch's arithmetic in 64 bits: in 32 these counts wrap to a negative grid
    status = q.raw_status("qtip_mx_matmul", 256, 256, m, 256, 256, n, 32, 256, q.QTIP_OUT_F32, None)
    assert status == CONFIG and "threads" in q.last_error_detail()


def test_expert_matmul_and_layer_refusals(plan):
    w = q.make_mx_weights(*[256] * 6)

    def call(part=q.QTIP_MX_PASS_GATE_UP, weights=w, a=256, sa=256, off=256, sp=256, n=4, out=256, kind=0):
        return q.raw_status("qtip_mx_expert_matmul", plan, part, None if weights is None else ctypes.byref(weights), a,
                            sa, off, sp, n, out, kind, None)
    assert call(part=2) == ARG and call(weights=None) == ARG and call(kind=2) == ARG
    for name in ("a", "sa", "off", "sp", "out"):
        assert call(**{name: None}) == ARG
    assert call(a=264) == ARG and call(sa=258) == ARG and call(out=264) == ARG
    assert call(n=0) == CONFIG and call(n=65) == CONFIG
    down_only = q.make_mx_weights(codes_down=256, scales_down=256)
    assert call(weights=down_only) == ARG and "weight" in q.last_error_detail()
    assert call(part=q.QTIP_MX_PASS_DOWN, weights=q.make_mx_weights(*[256] * 4)) == ARG
    assert call(weights=q.make_mx_weights(264, 256, 256, 256)) == ARG
    assert call(weights=q.make_mx_weights(256, 257, 256, 256)) == ARG

    size = q.qtip_mx_moe_workspace_bytes(plan)
    assert size > 0 and q.qtip_mx_moe_workspace_bytes(None) == 0
    layer = lambda weights=w, x=256, lg=256, n=4, out=256, ws=256, s=size: q.raw_status(
        "qtip_mx_moe_forward", plan, None if weights is None else ctypes.byref(weights), None, x, lg, n, out, ws, s,
        None)
    assert layer(weights=down_only) == ARG and layer(weights=None) == ARG
    assert layer(x=None) == ARG and layer(lg=None) == ARG and layer(out=None) == ARG and layer(ws=None) == ARG
    assert layer(x=264) == ARG and layer(out=264) == ARG and layer(ws=384) == ARG and layer(s=size - 1) == ARG
    assert layer(n=0) == CONFIG and layer(n=65) == CONFIG


def test_tensors_in_host_memory_are_refused(plan):
    torch = pytest.importorskip("torch")
    t = torch.zeros(1 << 16, dtype=torch.uint8)
    f = torch.zeros(64)
    gate, w = q.make_gate(), q.make_weights(*[256] * 7)
    mw = q.make_mx_weights(*[256] * 6)
    for call in (lambda: q.qtip_mx_matmul(t, t, 1, t, t, 1, 32, t, q.QTIP_OUT_F32),
                 lambda: q.qtip_mx_matmul(256, 256, 1, 256, 256, 1, 32, t, q.QTIP_OUT_F32),
                 lambda: q.qtip_mx_quantize(f, q.QTIP_MX_SRC_F32, 1, 64, 64, 0, 256, 256),
                 lambda: q.qtip_mx_quantize(256, q.QTIP_MX_SRC_F32, 1, 64, 64, 0, 256, 256, f),
                 lambda: q.qtip_mx_expert_matmul(plan, 0, mw, t, 256, 256, 256, 1, 256, 0),
                 lambda: q.qtip_moe_gate_route(plan, gate, f, 1, 256, 256, 256, 256, 256, None, None, 256, 1 << 20),
                 lambda: q.qtip_moe_gate_route(plan, q.make_gate(bias=f), 256, 1, 256, 256, 256, 256, 256, None, None,
                                               256, 1 << 20),
                 lambda: q.qtip_moe_forward_gated(plan, w, gate, t, 256, 1, 256, 256, 1 << 30),
                 lambda: q.qtip_mx_moe_forward(plan, mw, None, 256, f, 1, 256, 256, 1 << 30)):
        with pytest.raises(q.QtipError) as ei:
            call()
        assert ei.value.status == ARG and ("GPU memory" in str(ei.value) or "device" in str(ei.value))


@pytest.fixture
def gpu_arrays(monkeypatch):
    """torch, a maker of tensors that pass for arrays of GPU 0, and the list of calls that the binding lets through: none
    reaches the library."""
    torch = pytest.importorskip("torch")
    binding = q._binding
    real, calls = q.lib(), []

    class Array(torch.Tensor):
        place = 0

        def get_device(self):
            return self.place

    class Library:
        def __getattr__(self, name):
            if name in ("qtip_status_string", "qtip_last_error_detail", "qtip_moe_plan_destroy"):
                return getattr(real, name)
            return lambda *args: calls.append((name, args)) or q.QTIP_OK

    binding._find_torch()
    monkeypatch.setattr(binding, "_get_device", lambda: 0)
    monkeypatch.setattr(binding, "_stream", lambda stream: None)
    monkeypatch.setattr(binding, "lib", lambda: Library())

    def array(*shape, dtype="uint8", device=0):
        t = torch.zeros(shape, dtype=getattr(torch, dtype)).as_subclass(Array)
        t.place = device
        return t
    return torch, array, calls


def refusals(call, good, bad, calls):
    """`good` arguments go through; with each of `bad` in one's place the call is refused, naming it."""
    call(**good)
    assert len(calls) == 1
    for name, value in bad:
        args = dict(good, **{name: value()})
        with pytest.raises(q.QtipError) as ei:
            call(**args)
        assert ei.value.status == ARG and name in str(ei.value), (name, str(ei.value))
    assert len(calls) == 1


def test_gate_route_takes_whole_arrays_of_its_types_only(gpu_arrays):
    torch, array, calls = gpu_arrays
    n, E, k = 5, 256, 6
    plan = q._binding.Plan(0, q.make_desc(E, k, 4096, 2048, 64))
    i32 = lambda *s: array(*s, dtype="int32")
    f32 = lambda *s: array(*s, dtype="float32")
    good = dict(bias=f32(E), logits=f32(n, E), topk_idx=i32(n, k), topk_w=f32(n, k), counts=i32(E), offsets=i32(E + 1),
                sorted_pair=i32(n * k), tile_map=i32(n * k, 3), n_tiles=i32(1), workspace=array(512))
    call = lambda bias, workspace, **a: q.qtip_moe_gate_route(
        plan, q.make_gate(bias=bias), n_tokens=n, workspace=workspace, workspace_bytes=512, **a)
    bad = [(name, lambda t=t: t.reshape(-1)[:-1].contiguous()) for name, t in good.items()]        # one short
    bad += [(name, lambda t=t: t.half() if t.dtype == torch.float32 else t.long())                 # another type
            for name, t in good.items() if name != "workspace"]
    bad += [(name, lambda t=t: array(*t.shape, dtype=str(t.dtype)[6:], device=1)) for name, t in good.items()]
    bad += [("logits", lambda: f32(E, n).t()), ("logits", lambda: torch.zeros(n, E)),
            ("bias", lambda: f32(2 * E)[::2]), ("bias", lambda: torch.zeros(E)), ("topk_w", lambda: i32(n, k))]
    refusals(call, good, bad, calls)


def test_gated_layers_take_whole_arrays_of_their_types_only(gpu_arrays):
    torch, array, calls = gpu_arrays
    n, E, k, H, I = 5, 8, 2, 256, 128
    for out_dtype, out_type in ((q.QTIP_OUT_F32, "float32"), (q.QTIP_OUT_BF16, "bfloat16")):
        plan = q._binding.Plan(0, q.make_desc(E, k, H, I, 64, out_dtype=out_dtype))
        good = dict(bias=array(E, dtype="float32"), x_bf16=array(n, H, dtype="bfloat16"),
                    logits=array(n, E, dtype="float32"), out=array(n, H, dtype=out_type), workspace=array(512))
        bad = [(name, lambda t=t: t.reshape(-1)[:-1].contiguous()) for name, t in good.items()]
        bad += [("x_bf16", lambda: array(n, H, dtype="float16")), ("x_bf16", lambda: array(n, H, dtype="float32")),
                ("logits", lambda: array(n, 2 * E, dtype="bfloat16")), ("bias", lambda: array(2 * E, dtype="bfloat16")),
                ("out", lambda: array(n, H, dtype="float16")), ("out", lambda: array(n, H, dtype="float64")),
                ("out", lambda: array(n, H, dtype=out_type, device=1))]
        w = q.make_weights(*[256] * 7)
        refusals(lambda bias, **a: q.qtip_moe_forward_gated(plan, w, q.make_gate(bias=bias), n_tokens=n,
                                                            workspace_bytes=512, **a), good, bad, calls)
        calls.clear()
        names = ("codes_gate", "scales_gate", "codes_up", "scales_up", "codes_down", "scales_down")
        good.update((name, array(E * H * I // (32 if "scales" in name else 2))) for name in names)
        bad += [(name, lambda name=name: good[name][:-1].contiguous()) for name in names]
        bad += [(name, lambda name=name: good[name].float()) for name in names]
        bad += [("codes_up", lambda: array(E * H * I // 2, device=1)), ("scales_down", lambda: array(E * H * I)[::2]),
                ("codes_down", lambda: torch.zeros(E * H * I // 2, dtype=torch.uint8))]
        refusals(lambda bias, x_bf16, logits, out, workspace, **w: q.qtip_mx_moe_forward(
            plan, q.make_mx_weights(**w), q.make_gate(bias=bias), x_bf16, logits, n, out, workspace, 512), good, bad, calls)
        calls.clear()
        q.qtip_mx_moe_forward(plan, q.make_mx_weights(*[256] * 6), None, good["x_bf16"].view(torch.int16), 256, n, 256,
                              256, 512)          # addresses, and 16-bit patterns, as they come
        assert len(calls) == 1
        calls.clear()


@pytest.mark.parametrize("part", [q.QTIP_MX_PASS_GATE_UP, q.QTIP_MX_PASS_DOWN])
def test_expert_pass_takes_whole_arrays_of_its_types_only(gpu_arrays, part):
    torch, array, calls = gpu_arrays
    n, E, k, H, I = 5, 8, 2, 256, 128
    plan = q._binding.Plan(0, q.make_desc(E, k, H, I, 64))
    rows, cols, width = (n, H, I) if part == q.QTIP_MX_PASS_GATE_UP else (n * k, I, H)
    good = dict(a_codes=array(rows, cols // 2), a_scales=array(rows, cols // 32), offsets=array(E + 1, dtype="int32"),
                sorted_pair=array(n * k, dtype="int32"), out=array(n * k, width, dtype="bfloat16"))
    own = ("gate", "up") if part == q.QTIP_MX_PASS_GATE_UP else ("down",)
    weights = {f"{what}_{name}": array(E * H * I // (2 if what == "codes" else 32))
               for name in own for what in ("codes", "scales")}
    good.update(weights)
    bad = [(name, lambda t=t: t.reshape(-1)[:-1].contiguous()) for name, t in good.items()]
    bad += [(name, lambda t=t: array(*t.shape, dtype=str(t.dtype)[6:], device=1)) for name, t in good.items()]
    bad += [("offsets", lambda: array(E + 1, dtype="int64")), ("sorted_pair", lambda: array(n * k, dtype="int64")),
            ("a_codes", lambda: array(rows, cols, dtype="int32")), ("out", lambda: array(n * k, width, dtype="float32"))]

    def call(a_codes, a_scales, offsets, sorted_pair, out, **w):
        q.qtip_mx_expert_matmul(plan, part, q.make_mx_weights(**w), a_codes, a_scales, offsets, sorted_pair, n, out,
                                q.QTIP_OUT_BF16)
    refusals(call, good, bad, calls)
    calls.clear()
    call(**dict(good, **{name: array(1) for name in (f"{w}_{m}" for w in ("codes", "scales") for m in
                                                     ("gate", "up", "down") if m not in own)}))   # not this pass's
    assert len(calls) == 1


def test_dense_mx_calls_take_arrays_of_their_types_only(gpu_arrays):
    torch, array, calls = gpu_arrays
    for kind, name, other in ((q.QTIP_MX_SRC_BF16, "bfloat16", "float16"), (q.QTIP_MX_SRC_F16, "float16", "bfloat16"),
                              (q.QTIP_MX_SRC_F32, "float32", "int32")):
        good = dict(src=array(4, 80, dtype=name)[:, :64], codes=array(4, 32), scales=array(4, 2),
                    values=array(4, 64, dtype=name))
        bad = [("src", lambda: array(4, 80, dtype=other)), ("src", lambda: array(4 * 80 - 17, dtype=name)),
               ("src", lambda: array(4, 80, dtype=name, device=1)), ("values", lambda: array(4, 64, dtype=other)),
               ("codes", lambda: array(4, 32, dtype="int32")), ("scales", lambda: array(7))]
        refusals(lambda src, **a: q.qtip_mx_quantize(src, kind, 4, 64, 80, q.QTIP_MX_SCALE_FLOOR, **a), good, bad, calls)
        calls.clear()
    for kind, name, other in ((q.QTIP_OUT_BF16, "bfloat16", "float16"), (q.QTIP_OUT_F32, "float32", "int32")):
        good = dict(a_codes=array(3, 32), a_scales=array(3, 2), w_codes=array(5, 32), w_scales=array(5, 2),
                    out=array(3, 5, dtype=name))
        bad = [(key, lambda t=t: t.reshape(-1)[:-1].contiguous()) for key, t in good.items()]
        bad += [(key, lambda t=t: array(*t.shape, dtype=str(t.dtype)[6:], device=1)) for key, t in good.items()]
        bad += [("out", lambda: array(3, 5, dtype=other)), ("w_scales", lambda: array(5, 2, dtype="float32"))]
        refusals(lambda a_codes, a_scales, w_codes, w_scales, out: q.qtip_mx_matmul(
            a_codes, a_scales, 3, w_codes, w_scales, 5, 64, out, kind), good, bad, calls)
        calls.clear()
