"""Both sides of the e4m3 entry points' size limits.  They are decided on the host, and the sizes inside them meet a
later refusal, so that no call here gets as far as a device."""
import ctypes

import pytest

import trellis_quantized_moe_expert_amd as q

ARG, CONFIG = q.QTIP_ERR_INVALID_ARG, q.QTIP_ERR_INVALID_CONFIG


@pytest.mark.parametrize("hidden,inter", [((1 << 23) - 128, 128), (1 << 23, 128), (17_000_064, 128), (34_000_000, 128),
                                          (128, (1 << 23) - 128), (128, 1 << 23), (128, 34_200_064)])
def test_expert_passes_refuse_more_inputs_than_a_tile_can_address(hidden, inter):
    # 128 rows of a matrix of 17000064 inputs are past the 2^31 bytes of a buffer: rows behind them would count as zeros
    plan = q.qtip_moe_plan_for_arch(q.make_desc(1, 1, hidden, inter, 1), "gfx950")
    w = q.make_f8_weights(*[256] * 6)
    size = q.qtip_f8_moe_workspace_bytes(plan)

    def expert(part, n):
        return q.raw_status("qtip_f8_expert_matmul", plan, part, ctypes.byref(w), 256, 256, 256, 256, n, 256,
                            q.QTIP_OUT_F32, None, None)

    # without a token a call that passes is refused for that
    for part, inputs, name in ((q.QTIP_F8_PASS_GATE_UP, hidden, "hidden"), (q.QTIP_F8_PASS_DOWN, inter, "inter")):
        if inputs < 1 << 23:
            assert expert(part, 0) == CONFIG
        else:
            for n in (0, 1):
                assert expert(part, n) == ARG and name in q.last_error_detail()
    layer = lambda n: q.raw_status("qtip_f8_moe_forward", plan, ctypes.byref(w), None, 256, 256, 256, n, 256, 256, size,
                                   None)
    if max(hidden, inter) < 1 << 23:
        assert layer(0) == CONFIG
    else:
        for n in (0, 1):
            assert layer(n) == ARG and "2^23" in q.last_error_detail()
    q.qtip_moe_plan_destroy(plan)


def test_quantisation_of_128_rows_a_block_takes_fewer_than_2_24_blocks():
    def detail(rows, cols):
        # codes that are not aligned: what the sizes let through is refused for that
        assert q.raw_status("qtip_f8_quantize", 256, q.QTIP_F8_BF16, rows, cols, cols, 128, q.QTIP_F8_SCALE_AMAX, 264, 256,
                            None) == ARG
        return q.last_error_detail()
    for rows, cols in ((1 << 29, 1), ((1 << 29) + 130, 128), (2 ** 31 - 128, 1), ((1 << 18) - 128, 1 << 20)):
        assert "aligned" in detail(rows, cols), (rows, cols)
    for rows, cols in ((2 ** 31 - 127, 1), (2 ** 31 - 1, 128), (1 << 18, 1 << 20)):
        assert "blocks" in detail(rows, cols), (rows, cols)
