"""The gate's and MXFP4's oracles against hand-worked values and independent formulas."""
import math

import numpy as np
import pytest

from oracle import gate, mx, routing


def test_softmax_gate_without_groups_is_the_plain_routing():
    rng = np.random.default_rng(0)
    logits = rng.standard_normal((40, 24)).astype(np.float32)
    idx, w = gate.route(logits, None, 5)
    ref_idx, ref_w = routing.route_topk(logits, 5)   # softmax over the k chosen = renormalised softmax over all
    assert np.array_equal(idx, ref_idx)
    assert np.allclose(w, ref_w, rtol=1e-6)


def test_bias_moves_the_choice_but_not_the_weight():
    idx, w = gate.route_token([0.0, 1.0, 2.0, -1.0], [9.0, 0.0, 0.0, 0.0], 2, "sigmoid", renormalise=0)
    assert idx == [0, 2]
    assert w == pytest.approx([0.5, 1 / (1 + math.exp(-2.0))])


def test_groups_by_the_sum_of_two():
    # group values (top two): 0.5 + 0.5, 0.88 + 0.27, 0.73 + 0.73
    row = [0.0, 0.0, 2.0, -1.0, 1.0, 1.0]
    idx, _ = gate.route_token(row, None, 2, "sigmoid", num_groups=3, top_groups=1, group_top=2)
    assert idx == [4, 5]
    idx, _ = gate.route_token(row, None, 2, "sigmoid", num_groups=3, top_groups=1, group_top=1)
    assert idx == [2, 3]


def test_masked_experts_are_never_chosen():
    ninf, nan = -math.inf, math.nan
    assert gate.route_token([ninf, 1.0, nan, 0.0], None, 3) == ([1, 3, -1], pytest.approx(
        [1 / (1 + math.exp(-1.0)), 1 / (1 + math.exp(1.0)), 0.0]))
    assert gate.route_token([ninf] * 4, None, 2) == ([-1, -1], [0.0, 0.0])
    assert gate.route_token([3.0, 2.0, 1.0], [ninf, 0.0, nan], 2, "sigmoid")[0] == [1, -1]
    idx, w = gate.route_token([math.inf, 0.0, math.inf], None, 3, renormalise=0)
    assert idx == [0, 2, 1] and w == [0.5, 0.5, 0.0]


def test_shares_of_scores_at_the_end_of_fp64():
    # exp(-1) : 1 whatever lies above, down to scores of exp(-745)
    want = [1 / (1 + math.exp(-1.0)), 1 / (1 + math.e)]
    for gap in (0.0, 600.0, 709.0, 720.0, 744.0):
        row, bias = [40.0, -gap + 40.0, -gap + 39.0], [-math.inf, 2.0, 1.0]
        assert gate.route_token(row, bias, 2)[1] == pytest.approx(want, rel=1e-12)
        assert gate.route_token([-gap - 5.0, -gap - 6.0], None, 2, "sigmoid")[1] == (
            [0.0, 0.0] if gap > 740 else pytest.approx(want, rel=2e-2 if gap == 0 else 1e-12))
    assert gate.route_token([40.0, -706.0, -706.0], [-math.inf, 0.0, 0.0], 2)[1] == [0.0, 0.0]
    assert gate.route_token([math.inf, 3.0, 3.0], [-math.inf, 0.0, 0.0], 2)[1] == [0.0, 0.0]
    assert gate.route_token([-703.0, -701.0, -702.0], None, 2, "sigmoid")[0] == [1, 2]


def test_bins_leave_out_pairs_without_an_expert():
    counts, offsets, order = gate.bins(np.array([[2, 0], [-1, 2], [0, -1]]), 3)
    assert counts.tolist() == [2, 0, 2] and offsets.tolist() == [0, 2, 2, 4] and order.tolist() == [1, 4, 0, 3]


def test_quantise_hand_worked_block():
    v = np.zeros(32)
    v[:10] = [4.0, -0.25, 0.26, 0.75, -1.25, 2.5, 3.5, 5.0, 7.9, -0.0]
    codes, byte, values = mx.quantise_block(v, "floor")
    assert byte == 127                                  # amax 7.9: exponent 2, scale 2^0
    assert values[:10].tolist() == [4.0, -0.0, 0.5, 1.0, -1.0, 2.0, 4.0, 4.0, 6.0, -0.0]
    assert codes[:5].tolist() == [0x86, 0x21, 0x4A, 0x66, 0x87]
    _, byte, values = mx.quantise_block(v, "nearest")   # 7.9 >= 7: one step larger
    assert byte == 128 and values[8] == 8.0 and values[6] == 4.0 and values[4] == -1.0
    assert mx.quantise_block(np.where(v == 7.9, 6.99, v), "nearest")[1] == 127


@pytest.mark.parametrize("rule", ["floor", "nearest"])
def test_decode_inverts_quantise(rule):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((7, 70)) * np.exp2(rng.integers(-140, 120, (7, 70)).astype(float))
    x[0] = 0.0
    codes, scales, values = mx.quantise(x, rule)
    assert np.array_equal(mx.decode(codes, scales)[:, :70], values)
    assert np.all(mx.decode(codes, scales)[:, 70:] == 0)
    # the values are fixed points of the floor rule where amax stayed on the grid
    again = mx.quantise(values, rule)[2]
    assert np.array_equal(again, values)


def test_quantise_extremes():
    tiny = np.zeros(32)
    tiny[0] = 2.0 ** -130
    assert mx.quantise_block(tiny, "floor")[1] == 0
    bad = np.ones(32)
    bad[5] = np.inf
    codes, byte, values = mx.quantise_block(bad, "floor")
    assert byte == 255 and not codes.any() and np.isnan(values).all()
    assert np.isnan(mx.decode(codes, np.array([byte]))).all()
