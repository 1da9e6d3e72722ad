"""Routing with a gate on the GPU against the oracle: expert ids and bins exactly, weights within
the documented factor 1 +- 2^-21."""
import math

import numpy as np
import pytest

import trellis_quantized_moe_expert_amd as q
from gpu_util import say
from oracle import gate as oracle

pytestmark = pytest.mark.gpu

SCORES = {"softmax": q.QTIP_GATE_SOFTMAX, "sigmoid": q.QTIP_GATE_SIGMOID}


class Route:
    """A plan, a gate and outputs (filled with a mark) for batches of up to n tokens."""

    def __init__(self, E, k, n, bias=None, score="softmax", tiles=True, **gate):
        import torch
        self.E, self.k, self.n = E, k, n
        self.plan = q.qtip_moe_plan(q.make_desc(E, k, 128, 128, n), 0)
        self.bias = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
        self.gate = q.make_gate(score=SCORES[score], bias=self.bias, **gate)
        mark = lambda *s, dt=torch.int32: torch.full(s, -7, dtype=dt, device="cuda:0")
        self.out = dict(topk_idx=mark(n, k), topk_w=mark(n, k, dt=torch.float32), counts=mark(E), offsets=mark(E + 1),
                        sorted_pair=mark(n * k), tile_map=mark(n * k, 3) if tiles else None,
                        n_tiles=mark(1) if tiles else None)
        size = q.qtip_moe_gate_workspace_bytes(self.plan)
        self.ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda:0")

    def call(self, logits, n=None):
        o = self.out
        q.qtip_moe_gate_route(self.plan, self.gate, logits, n or logits.shape[0], o["topk_idx"], o["topk_w"],
                              o["counts"], o["offsets"], o["sorted_pair"], o["tile_map"], o["n_tiles"], self.ws,
                              self.ws.numel())

    def host(self):
        import torch
        torch.cuda.synchronize()
        return {k: None if v is None else v.cpu().numpy() for k, v in self.out.items()}

    def close(self):
        q.qtip_moe_plan_destroy(self.plan)


def check(got, idx, w, E, n, k):
    assert np.array_equal(got["topk_idx"].reshape(-1)[:n * k], idx.reshape(-1))
    err = np.abs(got["topk_w"].reshape(-1)[:n * k] - w.reshape(-1))
    assert np.all(err <= 2.0 ** -21 * np.abs(w.reshape(-1)) + 1e-45), float(err.max())
    counts, offsets, order = oracle.bins(idx, E)
    assert np.array_equal(got["counts"], counts)
    assert np.array_equal(got["offsets"], offsets)
    assert np.array_equal(got["sorted_pair"][:len(order)], order)
    assert np.all(got["sorted_pair"][len(order):] == -7)       # left as they were
    if got["tile_map"] is not None:
        tiles = [(e, int(offsets[e]) + s, min(16, int(counts[e]) - s)) for e in range(E)
                 for s in range(0, int(counts[e]), 16)]
        assert int(got["n_tiles"][0]) == len(tiles)
        assert np.array_equal(got["tile_map"][:len(tiles)].reshape(-1, 3), np.array(tiles, np.int32).reshape(-1, 3))


def run(logits, E, k, bias=None, tiles=True, **gate):
    import torch
    n = logits.shape[0]
    r = Route(E, k, n, bias, tiles=tiles, **gate)
    r.call(torch.from_numpy(logits).cuda())
    got = r.host()
    r.close()
    kw = {key: gate[key] for key in gate}
    idx, w = oracle.route(logits, bias, k, **kw)
    check(got, idx, w, E, n, k)


CASES = [
    # n, E, k, gate
    (1, 256, 8, dict(score="sigmoid", num_groups=8, top_groups=4, group_top=2, scale=2.5)),
    (1, 1, 1, dict()),
    (2, 8, 8, dict(score="sigmoid", renormalise=0)),
    (5, 64, 6, dict(num_groups=64, top_groups=9)),
    (7, 60, 5, dict(renormalise=0)),
    (33, 160, 6, dict(num_groups=8, top_groups=3, group_top=1, renormalise=0, scale=16.0)),
    (64, 7, 3, dict(score="sigmoid")),
    (65, 1024, 32, dict(score="sigmoid", num_groups=32, top_groups=5, group_top=2)),
    (100, 1000, 17, dict(num_groups=4, top_groups=2, group_top=2)),
    (129, 72, 4, dict(score="sigmoid", num_groups=24, top_groups=2, group_top=2)),
    (300, 256, 8, dict(score="sigmoid", num_groups=8, top_groups=8, group_top=2)),
    (1030, 96, 2, dict(num_groups=3, top_groups=1, group_top=2)),
    (513, 65, 4, dict(num_groups=5, top_groups=2)),
    (40, 320, 16, dict(score="sigmoid", num_groups=2, top_groups=1)),
    (2500, 33, 3, dict(score="sigmoid")),
    # each side of the kernels' own borders: tokens of one workgroup, of small workgroups, of one pass
    (16, 256, 4, dict(score="sigmoid")),
    (17, 256, 9, dict(score="sigmoid", num_groups=4, top_groups=2)),
    (16, 300, 33 - 1, dict()),
    (1024, 40, 8, dict(num_groups=2, top_groups=1)),
    (1025, 40, 9, dict(score="sigmoid")),
    (4097, 24, 4, dict(num_groups=3, top_groups=2, group_top=2)),
    (9000, 12, 1, dict(score="sigmoid")),
    (600, 260, 3, dict(score="sigmoid", num_groups=2, top_groups=1)),
    (33000, 8, 2, dict()),
    (8300, 272, 2, dict(score="sigmoid")),
]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("n,E,k,gate", CASES)
def test_gate_matches_the_oracle(n, E, k, gate, bias):
    rng = np.random.default_rng(1000 * n + E + bias)
    say(f"gate n={n} E={E} k={k} {gate} bias={bias}")
    b = (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None
    run(rng.standard_normal((n, E)).astype(np.float32), E, k, b, tiles=not bias, **gate)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(64, 6, 1), (64, 6, 8), (256, 8, 8), (40, 12, 4)])
def test_ties_go_to_the_lower_index(E, k, groups, score):
    rng = np.random.default_rng(E + k + groups)
    logits = np.round(rng.standard_normal((50, E)) * 1.2).astype(np.float32)
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    bias = np.round(2 * rng.standard_normal(E)).astype(np.float32) / 8
    say(f"gate ties E={E} k={k} groups={groups} {score}")
    for b in (None, bias):
        run(logits, E, k, b, score=score, num_groups=groups, top_groups=max(1, groups // 2), group_top=1 + groups // 8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_closer_than_fp32_resolves(score):
    # neighbouring fp32 logits: their sigmoids (and biased scores) agree to the last fp32 bit
    rng = np.random.default_rng(5)
    E = 64
    base = rng.uniform(1.0, 3.0, (200, 1)).astype(np.float32)
    steps = rng.permuted(np.tile(np.arange(E), (200, 1)), axis=1)
    logits = (base.view(np.int32) + steps.astype(np.int32)).view(np.float32)
    say(f"gate close scores {score}")
    run(logits, E, 6, None, score=score)
    run(logits, E, 6, np.full(E, 0.25, np.float32), score=score)
    run(logits, E, 6, None, score=score, num_groups=8, top_groups=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_experts_and_empty_rows(score, groups):
    rng = np.random.default_rng(11)
    E, k, n = 32, 6, 70
    logits = rng.standard_normal((n, E)).astype(np.float32)
    logits[rng.random((n, E)) < 0.7] = -np.inf
    logits[3] = -np.inf                                # nothing left
    logits[4] = np.nan
    logits[5] = np.finfo(np.float32).min               # the type's lowest value is a number
    logits[6, :7] = np.nan
    logits[7, 5:9] = np.inf
    logits[8] = 3.4e38
    logits[9, 1:] = -np.inf
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    bias[[2, 30]] = -np.inf
    bias[7] = np.nan
    bias[9] = np.inf
    say(f"gate masks {score} groups={groups}")
    for b in (None, bias):
        for renorm in (0, 1):
            run(logits, E, k, b, score=score, num_groups=groups, top_groups=max(1, groups // 2), group_top=2 - (groups == 1),
                renormalise=renorm)


def test_extreme_logits():
    rng = np.random.default_rng(12)
    logits = (rng.standard_normal((64, 48)) * 60).astype(np.float32)
    say("gate extreme logits")
    run(logits, 48, 4, None, score="sigmoid")
    run(logits, 48, 4, None, score="softmax", renormalise=0)
    run((logits * 20).astype(np.float32), 48, 4, (0.01 * rng.standard_normal(48)).astype(np.float32), score="softmax")


# (E, k, groups, copies of the rows): one workgroup, a wave or a quarter of one a token, 4 to 32 experts a
# lane, lists of 8 and of 32 (two choices a lane)
LOW = [(48, 2, 1, 1), (48, 5, 4, 1), (48, 5, 4, 4), (240, 24, 1, 200), (256, 8, 8, 200), (300, 5, 2, 3),
       (1000, 9, 1, 3)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,copies", LOW)
def test_weights_of_scores_at_the_end_of_fp64(E, k, groups, copies, score):
    # the experts that can be chosen lie `gap` below the softmax's largest logit (a sigmoid: below 0); the
    # bias takes the loud one out and makes the choice, the scores being far smaller
    rng = np.random.default_rng(E + k)
    gaps = [0, 300, 484, 486, 700, 702, 705, 708, 709, 712, 720, 735, 743, 746, 800, 2e5]
    near = rng.uniform(-2.0, 0.0, (len(gaps), E)).astype(np.float32)
    near[5] = 0.0                                      # equal scores
    near[np.arange(len(gaps)), rng.integers(1, E, len(gaps))] = -np.inf
    logits = (near - np.array(gaps, np.float32)[:, None]).astype(np.float32)
    if score == "softmax":
        logits += 90.0
        logits[:, 0] = 90.0
    bias = rng.permutation(E).astype(np.float32) / 64
    bias[0] = -np.inf
    say(f"gate low scores E={E} k={k} groups={groups} {score}")
    for renorm in (1, 0):
        run(np.tile(logits, (copies, 1)), E, k, bias, score=score, num_groups=groups, top_groups=max(1, groups // 2),
            renormalise=renorm, scale=2.5)
    lone = np.full((3, E), -np.inf, np.float32)        # one expert left, and none; the loud one infinite
    lone[0, 0], lone[0, 3] = 0.0, -730.0
    lone[1, 0] = 0.0
    lone[2, 0], lone[2, 1:4] = np.inf, 5.0
    run(lone, E, k, bias, score=score)


@pytest.mark.parametrize("groups", [1, 4])
def test_order_of_low_sigmoids(groups):
    # scores of 4e-305 to 7e-308 are fp64 numbers: their order decides, among groups too
    rng = np.random.default_rng(40 + groups)
    E = 64
    logits = (-701.0 - rng.permuted(np.tile(np.arange(E) * 0.1, (40, 1)), axis=1)).astype(np.float32)
    say(f"gate order of low sigmoids, groups={groups}")
    for n in (40, 5):
        for group_top in (1, 2):
            run(logits[:n], E, 6, None, score="sigmoid", num_groups=groups, top_groups=max(1, groups // 2),
                group_top=group_top)


def test_fewer_tokens_than_the_plan_and_rows_behind_left_alone():
    import torch
    rng = np.random.default_rng(2)
    r = Route(64, 4, 300, score="sigmoid")
    logits = rng.standard_normal((120, 64)).astype(np.float32)
    say("gate n below the plan's")
    r.call(torch.from_numpy(logits).cuda())
    got = r.host()
    idx, w = oracle.route(logits, None, 4, score="sigmoid")
    check(got, idx, w, 64, 120, 4)
    assert np.all(got["topk_idx"][120:] == -7) and np.all(got["topk_w"][120:] == -7)
    r.close()


def test_skewed_batch_fills_one_bin():
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((3000, 16)).astype(np.float32)
    logits[:, 5] += 9.0
    say("gate one hot expert")
    run(logits, 16, 2, None, score="sigmoid")


def test_blocks_of_more_pairs_than_a_wave_keeps():
    # 512 blocks of 320 tokens, 640 pairs a wave; the oracle chooses for the 700 different rows
    import torch
    n, E, k = 140000, 64, 32
    rng = np.random.default_rng(11)
    rows = rng.standard_normal((700, E)).astype(np.float32)
    rows[::7, rng.permutation(E)[:40]] = -np.inf                # 24 experts left: slots stay empty
    say(f"gate n={n} E={E} k={k}, many pairs a block")
    r = Route(E, k, n, score="sigmoid", tiles=False)
    r.call(torch.from_numpy(rows).cuda().repeat(n // 700, 1))
    got = r.host()
    r.close()
    idx, w = oracle.route(rows, None, k, score="sigmoid")
    check(got, np.tile(idx, (n // 700, 1)), np.tile(w, (n // 700, 1)), E, n, k)


def test_gate_in_a_graph_and_on_another_stream():
    import torch
    rng = np.random.default_rng(8)
    E, k, n = 256, 8, 700
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    kw = dict(score="sigmoid", num_groups=8, top_groups=4, group_top=2, scale=2.5)
    batches = [rng.standard_normal((n, E)).astype(np.float32) for _ in range(3)]
    refs = [oracle.route(b, bias, k, **kw) for b in batches]
    a, other = Route(E, k, n, bias, **kw), Route(E, k, n, bias, **kw)
    buf = torch.from_numpy(batches[0]).cuda()
    dev = [torch.from_numpy(b).cuda() for b in batches]
    say("gate captured")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a.call(buf)                                     # another stream, and the witness outside capture
        s.synchronize()
        check(a.host(), *refs[0], E, n, k)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a.call(buf)
    torch.cuda.synchronize()
    for i in (1, 2, 0, 1):
        buf.copy_(dev[i])
        other.call(dev[(i + 1) % 3])                    # eager work between replays, its own workspace
        torch.cuda.synchronize()
        g.replay()
        check(a.host(), *refs[i], E, n, k)
        check(other.host(), *refs[(i + 1) % 3], E, n, k)
    a.close()
    other.close()


def test_binding_refuses_host_and_strided_tensors():
    import torch
    r = Route(64, 4, 8)
    with pytest.raises(q.QtipError):
        r.call(torch.zeros(8, 64))
    with pytest.raises(q.QtipError):
        r.call(torch.zeros(64, 8, device="cuda:0").t())
    r.close()
