"""Random MXFP4 operands, error bounds and routed batches for the MXFP4 tests."""
import numpy as np

from oracle import gate as gate_oracle
from oracle import mx


def packed(rng, rows, cols, lo=118, hi=130):
    """Uniform random codes, scale bytes in [lo, hi)."""
    return (rng.integers(0, 256, (rows, cols // 2)).astype(np.uint8),
            rng.integers(lo, hi, (rows, cols // 32)).astype(np.uint8))


def sum_bound(a, w):
    """Bound of |fp32 sum - exact| for sums over K of products a w: an instruction adds 128 products
    (exact: 6 x 6 x 2^s has few bits) to the running sum, in at most 8 partial sums of 32 with a last
    bit of 2^-23 of the largest magnitude met, S = sum |a w|; K / 32 + 16 such steps cover the
    instructions and the joining of the waves' sums."""
    steps = a.shape[1] / 32 + 16
    return steps * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)


def rounded(bound, ref, dtype):
    """The bound with the output's rounding (half a step) added."""
    return bound + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * (np.abs(ref) + bound) + 1e-38


def bins_of(rng, n, E, k, skew=False, holes=0.0):
    """A batch's expert ids [n][k] (distinct per token; a share of them -1) and bins."""
    idx = np.stack([rng.permutation(E)[:k] for _ in range(n)]).astype(np.int32)
    if skew:
        idx[:, 0] = np.where((idx == E // 2).any(1), idx[:, 0], E // 2)
    if holes:
        idx[rng.random(idx.shape) < holes] = -1
    counts, offsets, order = gate_oracle.bins(idx, E)
    return idx, counts, offsets, order


def values(codes, scales):
    return mx.decode(codes, scales)
