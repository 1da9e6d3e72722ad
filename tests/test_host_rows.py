"""Rows whose elements do not lie side by side: every call that takes rows of a wider tensor refuses them."""
import trellis_quantized_moe_expert_amd as q
from test_host_gate_mx import gpu_arrays, refusals  # noqa: F401  (a fixture)


def test_rows_of_elements_that_lie_apart_are_refused(gpu_arrays):  # noqa: F811
    torch, array, calls = gpu_arrays
    bf16 = lambda *s: array(*s, dtype="bfloat16")
    f32 = lambda *s: array(*s, dtype="float32")
    every_other = lambda: bf16(6, 160)[:, ::2]
    turned = lambda: bf16(160, 160).t()
    good = dict(src=bf16(6, 160)[:, :72], codes=array(6, 80), scales=f32(6, 1))
    for high in (1, 128):
        refusals(lambda src, **a: q.qtip_f8_quantize(src, q.QTIP_F8_BF16, 6, 72, 160, high, q.QTIP_F8_SCALE_AMAX, **a),
                 good, [("src", every_other), ("src", turned), ("src", lambda: bf16(2000)[::2])], calls)
        calls.clear()
    good = dict(src=bf16(6, 160)[:, :64], codes=array(6, 32), scales=array(6, 2))
    refusals(lambda src, **a: q.qtip_mx_quantize(src, q.QTIP_MX_SRC_BF16, 6, 64, 160, q.QTIP_MX_SCALE_FLOOR, **a), good,
             [("src", every_other), ("src", turned)], calls)
    calls.clear()
    good = dict(x=bf16(6, 160)[:, :72], residual=bf16(6, 160)[:, 8:80], residual_out=bf16(6, 160)[:, :72], weight=bf16(72),
                codes=array(6, 80), scales=f32(6, 1))
    refusals(lambda x, residual, residual_out, weight, codes, scales: q.qtip_f8_rms_norm(
        x, q.QTIP_F8_BF16, 6, 72, 160, residual, 160, residual_out, weight, q.QTIP_F8_BF16, 1e-6, q.QTIP_F8_SCALE_AMAX,
        codes, scales), good, [(name, make) for name in ("x", "residual", "residual_out") for make in (every_other, turned)],
        calls)
    calls.clear()
    # one element a row, the rows of an inner dimension, and a flat buffer are as they were
    q.qtip_f8_quantize(bf16(6, 160)[:, 3], q.QTIP_F8_BF16, 6, 1, 160, 1, 0, array(6, 16), f32(6, 1))
    q.qtip_f8_quantize(bf16(6, 160)[:, 3:4], q.QTIP_F8_BF16, 6, 1, 160, 1, 0, array(6, 16), f32(6, 1))
    q.qtip_f8_quantize(bf16(2, 3, 160)[:, :, :72], q.QTIP_F8_BF16, 6, 72, 160, 1, 0, array(6, 80), f32(6, 1))
    q.qtip_f8_quantize(bf16(6, 5, 32)[:, :3], q.QTIP_F8_BF16, 6, 96, 160, 1, 0, array(6, 96), f32(6, 1))
    q.qtip_f8_quantize(bf16(1000), q.QTIP_F8_BF16, 6, 72, 160, 1, 0, array(6, 80), f32(6, 1))
    assert len(calls) == 5
