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
