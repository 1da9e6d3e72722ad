"""Refusals of the e4m3 entry points: every one is decided on the host, before any device work, so plain
integers stand for device addresses here."""
import ctypes
import math

import pytest

import trellis_quantized_moe_expert_amd as q
from test_host_gate_mx import gpu_arrays, refusals  # noqa: F401  (a fixture)

V4 = dict(num_experts=256, top_k=6, hidden=4096, inter=2048, max_tokens=64)
ARG, CONFIG = q.QTIP_ERR_INVALID_ARG, q.QTIP_ERR_INVALID_CONFIG


@pytest.fixture
def plan():
    p = q.qtip_moe_plan_for_arch(q.make_desc(**V4), "gfx950")
    yield p
    q.qtip_moe_plan_destroy(p)


def test_quantize_refusals():
    def call(src=256, kind=q.QTIP_F8_BF16, rows=4, cols=64, stride=64, high=1, rule=q.QTIP_F8_SCALE_AMAX, codes=256,
             scales=256):
        return q.raw_status("qtip_f8_quantize", src, kind, rows, cols, stride, high, rule, codes, scales, None)
    assert call(src=None) == ARG and call(codes=None) == ARG and call(scales=None) == ARG
    assert call(kind=3) == ARG and call(kind=-1) == ARG and call(rule=2) == ARG and call(rule=-1) == ARG
    assert call(high=0) == ARG and call(high=64) == ARG and call(high=-128) == ARG
    assert call(rows=0) == CONFIG and call(cols=0) == CONFIG and call(rows=-1) == CONFIG
    assert call(stride=63) == ARG and call(stride=1 << 40) == ARG
    assert call(src=257) == ARG and call(src=258, kind=q.QTIP_F8_F32) == ARG
    assert call(codes=264) == ARG and call(scales=258) == ARG
    # 16 threads a block of a row, 256 a block of 128 rows: below 2^32
    assert call(rows=1 << 28, cols=128, stride=128) == ARG and call(rows=(1 << 28) - 15, cols=128, stride=128) == ARG
    assert call(rows=2 ** 31 - 1, cols=2 ** 31 - 1, stride=2 ** 31) == ARG
    assert call(rows=1 << 19, cols=1 << 19, stride=1 << 19, high=128) == ARG
    assert call(rows=2 ** 31 - 1, cols=200, stride=200, high=128) == ARG


def test_norm_refusals():
    def call(x=256, kind=q.QTIP_F8_BF16, rows=4, cols=64, stride=64, res=256, res_stride=64, out=256, w=256,
             w_kind=q.QTIP_F8_BF16, eps=1e-6, rule=q.QTIP_F8_SCALE_AMAX, codes=256, scales=256, values=256):
        return q.raw_status("qtip_f8_rms_norm", x, kind, rows, cols, stride, res, res_stride, out, w, w_kind, eps, rule,
                            codes, scales, values, None)
    for name in ("x", "w", "codes", "scales"):
        assert call(**{name: None}) == ARG
    assert call(res=None) == ARG and call(out=None) == ARG and "residual" in q.last_error_detail()
    assert call(kind=3) == ARG and call(w_kind=-1) == ARG and call(rule=2) == ARG
    for eps in (-1e-9, math.inf, math.nan):
        assert call(eps=eps) == ARG and "eps" in q.last_error_detail()
    assert call(rows=0) == CONFIG and call(cols=0) == CONFIG and call(cols=-4) == CONFIG
    assert call(rows=1 << 22) == ARG and call(cols=(1 << 30) + 1, stride=1 << 31, res_stride=1 << 31) == ARG
    assert call(stride=63) == ARG and call(res_stride=63) == ARG and call(stride=1 << 40) == ARG
    assert call(x=257) == ARG and call(res=257) == ARG and call(out=257) == ARG and call(w=257) == ARG
    assert call(x=258, kind=q.QTIP_F8_F32) == ARG and call(w=258, w_kind=q.QTIP_F8_F32) == ARG
    assert call(codes=264) == ARG and call(scales=258) == ARG and call(values=264) == ARG


def test_matmul_refusals():
    def call(a=256, sa=256, m=4, w=256, sw=256, n=32, k=64, out=256, kind=q.QTIP_OUT_F32):
        return q.raw_status("qtip_f8_matmul", a, sa, m, w, sw, n, k, out, kind, None)
    for name in ("a", "sa", "w", "sw", "out"):
        assert call(**{name: None}) == ARG
    assert call(kind=q.QTIP_OUT_E4M3) == ARG and call(kind=3) == ARG and call(k=40) == ARG
    assert call(m=0) == CONFIG and call(n=0) == CONFIG and call(k=0) == CONFIG and call(m=-4) == CONFIG
    assert call(a=264) == ARG and call(w=264) == ARG and call(out=264) == ARG and call(sa=257) == ARG
    assert call(sw=258) == ARG and call(k=1 << 23) == ARG
    assert call(m=1 << 30, k=128) == ARG and call(n=1 << 30, k=128) == ARG
    assert call(m=1 << 20, n=1 << 20, k=32) == ARG


@pytest.mark.parametrize("m,n", [(1, 1 << 28), (1, 2 ** 31 - 1), (16, 2 ** 31 - 16), (17, 2 ** 31 - 1), (2 ** 31 - 1, 1),
                                 (2 ** 31 - 1, 16), (2 ** 31 - 255, 300), (511, 2 ** 31 - 1), (1 << 19, (1 << 21) - 256)])
def test_products_past_2_32_threads_are_refused(m, n):
    for kind in (q.QTIP_OUT_F32, q.QTIP_OUT_BF16):
        status = q.raw_status("qtip_f8_matmul", 256, 256, m, 256, 256, n, 16, 256, kind, None)
        assert status == CONFIG and "threads" in q.last_error_detail()


def test_expert_matmul_and_layer_refusals(plan):
    w = q.make_f8_weights(*[256] * 6)

    def call(part=q.QTIP_F8_PASS_GATE_UP, weights=w, a=256, sa=256, off=256, sp=256, n=4, out=256, kind=q.QTIP_OUT_BF16,
             so=None):
        return q.raw_status("qtip_f8_expert_matmul", plan, part, None if weights is None else ctypes.byref(weights), a,
                            sa, off, sp, n, out, kind, so, None)
    assert call(part=2) == ARG and call(weights=None) == ARG and call(kind=3) == ARG
    for name in ("a", "sa", "off", "sp", "out"):
        assert call(**{name: None}) == ARG
    assert call(a=264) == ARG and call(sa=258) == ARG and call(out=264) == ARG
    assert call(n=0) == CONFIG and call(n=65) == CONFIG
    assert call(kind=q.QTIP_OUT_E4M3) == ARG and "out_scales" in q.last_error_detail()
    assert call(so=256) == ARG and call(kind=q.QTIP_OUT_E4M3, so=258) == ARG
    assert call(part=q.QTIP_F8_PASS_DOWN, kind=q.QTIP_OUT_E4M3, so=256) == ARG
    down_only = q.make_f8_weights(codes_down=256, scales_down=256)
    assert call(weights=down_only) == ARG and "weight" in q.last_error_detail()
    assert call(part=q.QTIP_F8_PASS_DOWN, weights=q.make_f8_weights(*[256] * 4)) == ARG
    assert call(weights=q.make_f8_weights(264, 256, 256, 256)) == ARG
    assert call(weights=q.make_f8_weights(256, 257, 256, 256)) == ARG

    size = q.qtip_f8_moe_workspace_bytes(plan)
    assert size > 0 and q.qtip_f8_moe_workspace_bytes(None) == 0
    layer = lambda weights=w, gate=None, x=256, sx=256, lg=256, n=4, out=256, ws=256, s=size: q.raw_status(
        "qtip_f8_moe_forward", plan, None if weights is None else ctypes.byref(weights),
        None if gate is None else ctypes.byref(gate), x, sx, lg, n, out, ws, s, None)
    assert layer(weights=down_only) == ARG and layer(weights=None) == ARG
    for name in ("x", "sx", "lg", "out", "ws"):
        assert layer(**{name: None}) == ARG
    assert layer(x=264) == ARG and layer(sx=258) == ARG and layer(out=264) == ARG and layer(ws=384) == ARG
    assert layer(s=size - 1) == ARG and layer(gate=q.make_gate(score=7)) == ARG
    assert layer(n=0) == CONFIG and layer(n=65) == CONFIG


def test_e4m3_is_no_output_of_the_other_products(plan):
    mw = q.make_mx_weights(*[256] * 6)
    assert q.raw_status("qtip_mx_matmul", 256, 256, 4, 256, 256, 32, 64, 256, q.QTIP_OUT_E4M3, None) == ARG
    assert q.raw_status("qtip_mx_expert_matmul", plan, 0, ctypes.byref(mw), 256, 256, 256, 256, 4, 256,
                        q.QTIP_OUT_E4M3, None) == ARG
    with pytest.raises(q.QtipError):
        q.qtip_moe_plan_for_arch(q.make_desc(**V4, out_dtype=q.QTIP_OUT_E4M3), "gfx950")


def test_rows_and_strides_of_other_tensors_are_refused(gpu_arrays):  # noqa: F811
    torch, array, calls = gpu_arrays
    for kind, name, other in ((q.QTIP_F8_BF16, "bfloat16", "float16"), (q.QTIP_F8_F16, "float16", "bfloat16"),
                              (q.QTIP_F8_F32, "float32", "int32")):
        good = dict(src=array(130, 80, dtype=name)[:, :72], codes=array(130, 80), scales=array(2, 1, dtype="float32"))
        bad = [("src", lambda: array(130, 80, dtype=other)), ("src", lambda: array(130 * 80 - 9, dtype=name)),
               ("src", lambda: array(130, 80, dtype=name, device=1)), ("src", lambda: torch.zeros(130, 80)),
               ("codes", lambda: array(130, 80, dtype="int32")), ("codes", lambda: array(130 * 80 - 1)),
               ("scales", lambda: array(1, dtype="float32")), ("scales", lambda: array(4, dtype="bfloat16"))]
        refusals(lambda src, **a: q.qtip_f8_quantize(src, kind, 130, 72, 80, 128, q.QTIP_F8_SCALE_AMAX, **a), good, bad,
                 calls)
        calls.clear()
        good = dict(x=array(5, 160, dtype=name)[:, :130], residual=array(5, 140, dtype=name)[:, :130],
                    residual_out=array(5, 140, dtype=name), weight=array(130, dtype="float32"), codes=array(5, 144),
                    scales=array(5, 2, dtype="float32"), values=array(5, 130, dtype=name))
        bad = [(key, lambda key=key: array(5, 160, dtype=other)) for key in ("x", "residual", "residual_out", "values")]
        bad += [("weight", lambda: array(130, dtype="bfloat16")), ("weight", lambda: array(129, dtype="float32")),
                ("x", lambda: array(5 * 160 - 31, dtype=name)), ("residual", lambda: array(5 * 140 - 11, dtype=name)),
                ("residual_out", lambda: array(5, 140, dtype=name, device=1)), ("values", lambda: array(5, 129, dtype=name)),
                ("codes", lambda: array(5, 143)), ("scales", lambda: array(9, dtype="float32"))]
        refusals(lambda x, residual, residual_out, weight, **a: q.qtip_f8_rms_norm(
            x, kind, 5, 130, 160, residual, 140, residual_out, weight, q.QTIP_F8_F32, 1e-6, q.QTIP_F8_SCALE_AMAX, **a),
            good, bad, calls)
        calls.clear()
    # whole arrays: the same checks, residual and values present or not
    good = dict(x=array(5, 130, dtype="bfloat16"), residual=array(5, 130, dtype="bfloat16"),
                residual_out=array(5, 130, dtype="bfloat16"), weight=array(130, dtype="bfloat16"), codes=array(5, 144),
                scales=array(5, 2, dtype="float32"), values=array(5, 130, dtype="bfloat16"))
    bad = [(key, lambda t=t: t.reshape(-1)[:-1].contiguous()) for key, t in good.items()]
    bad += [(key, lambda t=t: array(*t.shape, dtype=str(t.dtype)[6:], device=1)) for key, t in good.items()]
    bad += [(key, lambda t=t: t.half()) for key, t in good.items()]
    norm = lambda x, weight, codes, scales, residual=None, residual_out=None, values=None: q.qtip_f8_rms_norm(
        x, q.QTIP_F8_BF16, 5, 130, 130, residual, 130 if residual is not None else 0, residual_out, weight, q.QTIP_F8_BF16,
        1e-6, q.QTIP_F8_SCALE_AMAX, codes, scales, values)
    refusals(norm, good, bad, calls)
    for left_out in ("values", "residual", "values residual"):
        calls.clear()
        drop = left_out.replace("residual", "residual residual_out").split()
        some = {key: t for key, t in good.items() if key not in drop}
        refusals(norm, some, [b for b in bad if b[0] in some], calls)
        args = calls[0][1]
        assert [args[i] for i in (0, 8, 12, 13)] == [good[k].data_ptr() for k in ("x", "weight", "codes", "scales")]
        assert (args[5] is None) == ("residual" in left_out) and (args[14] is None) == ("values" in left_out)
    calls.clear()
    f8 = getattr(torch, "float8_e4m3fn")
    q.qtip_f8_quantize(256, q.QTIP_F8_F32, 4, 128, 128, 1, 0, array(4, 128).view(f8), 256)   # codes as their values' type
    assert len(calls) == 1


@pytest.mark.parametrize("part", [q.QTIP_F8_PASS_GATE_UP, q.QTIP_F8_PASS_DOWN])
def test_expert_pass_takes_whole_arrays_of_its_types_only(gpu_arrays, part):  # noqa: F811
    torch, array, calls = gpu_arrays
    n, E, k, H, I = 5, 8, 2, 256, 128
    plan = q._binding.Plan(0, q.make_desc(E, k, H, I, 64))
    up = part == q.QTIP_F8_PASS_GATE_UP
    rows, cols, width = (n, H, I) if up else (n * k, I, H)
    f32 = lambda *s: array(*s, dtype="float32")
    good = dict(a_codes=array(rows, cols), a_scales=f32(rows, cols // 128), offsets=array(E + 1, dtype="int32"),
                sorted_pair=array(n * k, dtype="int32"), out=array(n * k, width) if up else f32(n * k, width))
    if up:
        good["out_scales"] = f32(n * k, width // 128)
    names = ("gate", "up") if up else ("down",)
    good.update((f"codes_{name}", array(E * H * I)) for name in names)
    good.update((f"scales_{name}", f32(E * H * I // 128 ** 2)) for name in names)
    bad = [(name, lambda t=t: t.reshape(-1)[:-1].contiguous()) for name, t in good.items()]
    bad += [(name, lambda t=t: array(*t.shape, dtype=str(t.dtype)[6:], device=1)) for name, t in good.items()]
    bad += [(name, lambda t=t: t.half()) for name, t in good.items()]

    def call(a_codes, a_scales, offsets, sorted_pair, out, out_scales=None, **w):
        q.qtip_f8_expert_matmul(plan, part, q.make_f8_weights(**w), a_codes, a_scales, offsets, sorted_pair, n, out,
                                q.QTIP_OUT_E4M3 if up else q.QTIP_OUT_F32, out_scales)
    refusals(call, good, bad, calls)


def test_layer_and_product_take_whole_arrays_of_their_types_only(gpu_arrays):  # noqa: F811
    torch, array, calls = gpu_arrays
    n, E, k, H, I = 5, 8, 2, 256, 128
    f32 = lambda *s: array(*s, dtype="float32")
    plan = q._binding.Plan(0, q.make_desc(E, k, H, I, 64, out_dtype=q.QTIP_OUT_BF16))
    good = dict(bias=f32(E), x_codes=array(n, H), x_scales=f32(n, H // 128), logits=f32(n, E),
                out=array(n, H, dtype="bfloat16"), workspace=array(512))
    good.update((f"codes_{m}", array(E * H * I)) for m in ("gate", "up", "down"))
    good.update((f"scales_{m}", f32(E * H * I // 128 ** 2)) for m in ("gate", "up", "down"))
    bad = [(name, lambda t=t: t.reshape(-1)[:-1].contiguous()) for name, t in good.items()]
    bad += [(name, lambda t=t: array(*t.shape, dtype=str(t.dtype)[6:], device=1)) for name, t in good.items()]
    bad += [("x_codes", lambda: array(n, H, dtype="bfloat16")), ("out", lambda: f32(n, H))]
    refusals(lambda bias, x_codes, x_scales, logits, out, workspace, **w: q.qtip_f8_moe_forward(
        plan, q.make_f8_weights(**w), q.make_gate(bias=bias), x_codes, x_scales, logits, n, out, workspace, 512),
        good, bad, calls)
    calls.clear()
    good = dict(a_codes=array(3, 144), a_scales=f32(3, 2), w_codes=array(130, 144), w_scales=f32(2, 2), out=f32(3, 130))
    bad = [(key, lambda t=t: t.reshape(-1)[:-1].contiguous()) for key, t in good.items()]
    bad += [(key, lambda t=t: array(*t.shape, dtype=str(t.dtype)[6:], device=1)) for key, t in good.items()]
    bad += [(key, lambda t=t: t.half()) for key, t in good.items()]
    refusals(lambda a_codes, a_scales, w_codes, w_scales, out: q.qtip_f8_matmul(
        a_codes, a_scales, 3, w_codes, w_scales, 130, 144, out, q.QTIP_OUT_F32), good, bad, calls)
