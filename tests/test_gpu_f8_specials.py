"""e4m3 on the GPU at the edges of its range: sizes past one launch, and what the 8-bit matrix instructions make of NaN,
extreme scales and single inputs."""
import numpy as np
import pytest

import trellis_quantized_moe_expert_amd as q
from f8_util import RULE, TYPE, dtype_of, norm_bound, packed, same, spread, within
from gpu_util import say
from oracle import f8
from test_gpu_f8 import Experts, check_norm, check_product, norm, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [2 ** 29 - 128, 2 ** 29 - 127, 2 ** 29 + 130])
def test_quantise_blocks_of_128_rows_past_one_launch(rows):
    # one column: 2^22 - 1 blocks are the most of a launch of 1024 threads a block
    import torch
    say(f"quantise {rows}x1 in blocks of 128 rows")
    part = 2 ** 14
    g = torch.Generator().manual_seed(9)
    base = (torch.randn(part, 1, generator=g) * torch.exp2(torch.randint(-9, 9, (part // 128, 1), generator=g).float())
            .repeat_interleave(128, dim=0)).to(torch.bfloat16)
    x = base.cuda().repeat(-(-rows // part), 1)[:rows]
    blocks = -(-rows // 128)
    codes = torch.full((rows + 2, 16), 0xA5, dtype=torch.uint8, device="cuda:0")
    scales = torch.full((blocks + 2,), -7.0, device="cuda:0")
    q.qtip_f8_quantize(x, TYPE["bf16"], rows, 1, 1, 128, RULE["amax"], codes, scales)
    torch.cuda.synchronize()
    want = f8.quantise(base.double().numpy(), "amax", 128)
    codes_of, scales_of = torch.from_numpy(want[0]).cuda(), torch.from_numpy(want[1][:, 0]).cuda()
    whole = rows // part
    for piece in codes[:whole * part].view(whole, part, 16).split(2 ** 12):
        assert bool((piece == codes_of).all())
    assert bool((scales[:whole * part // 128].view(whole, -1) == scales_of).all())
    # the rest: whole blocks, and a last one of few rows
    rest = rows - whole * part
    if rest:
        codes_of, scales_of = f8.quantise(base[:rest].double().numpy(), "amax", 128)
        assert np.array_equal(codes[whole * part:rows].cpu().numpy(), codes_of)
        assert np.array_equal(scales[whole * part // 128:blocks].cpu().numpy(), scales_of[:, 0])
    assert bool((codes[rows:] == 0xA5).all()) and bool((scales[blocks:] == -7.0).all())


# ---- bf16 products: the 8-bit matrix instructions ------------------------------------------------
# every tile of the dense product's bf16 results, by the workgroups that the sizes make
TILES = [(40, 300, 544), (300, 2056, 544), (290, 3500, 288), (683, 2056, 544), (1000, 2056, 160), (1281, 5001, 400),
         (1500, 4702, 1040), (4000, 4100, 64)]


@pytest.mark.parametrize("m,n,k", [(1, 200, 160)] + TILES)
def test_nan_reaches_its_own_bf16_outputs_only(m, n, k):
    say(f"bf16 product {m}x{n}x{k} with NaN blocks")
    rng = np.random.default_rng(m + n)
    a, w = packed(rng, m, k), packed(rng, n, k, 128)
    before = product(a, w, k, "bf16")
    assert np.all(np.isfinite(before))
    a[1][m - 1, -1] = np.nan                # the last block of the last row
    a[0][m // 2, 0] = 0xff                  # a code of the activations
    w[0][n // 2, k - 1] = 0x7f              # and of the weights
    w[1][-1, 0] = np.nan                    # the first block of the last rows
    after = product(a, w, k, "bf16")
    hit = np.zeros((m, n), bool)
    hit[m - 1] = hit[m // 2] = hit[:, n // 2] = hit[:, (n - 1) // 128 * 128:] = True
    assert np.all(np.isnan(after[hit]))
    assert np.array_equal(after[~hit], before[~hit])


@pytest.mark.parametrize("m,n,k", [(20, 40, 256), (300, 400, 256)] + TILES)
def test_bf16_products_of_extreme_scales(m, n, k):
    say(f"bf16 product {m}x{n}x{k} of extreme scales")
    rng = np.random.default_rng(m)
    check_product(packed(rng, m, k, 1, -126, -100), packed(rng, n, k, 128, 30, 100), "bf16")
    check_product(packed(rng, m, k, 1, 60, 100), packed(rng, n, k, 128, -126, -100), "bf16")


@pytest.mark.parametrize("m,n", [(16, 16)] + [t[:2] for t in TILES])
def test_bf16_product_one_chunk_at_a_time(m, n):
    # 16 nonzero inputs at a time, all of their products multiples of 2^-8 of exponents -2 to 0: nothing is cut, the sums
    # are exact, and the result is the exact one rounded once
    import torch
    say(f"bf16 product chunk by chunk {m}x{n}")
    rng = np.random.default_rng(4)
    k = 656                                  # 128 x 256 tiles in three stages want more than 512
    for c in range(0, k, 16) if m < 300 else (0, 112, 128, 384, 640):
        a, w = packed(rng, m, k), packed(rng, n, k, 128)
        for codes in (a[0], w[0]):
            small = rng.integers(0x30, 0x40, codes.shape)          # 0.5 .. 1.875
            codes[:] = 0
            codes[:, c:c + 16] = small[:, c:c + 16]
        for scales in (a[1], w[1]):
            scales[:] = np.exp2(rng.integers(-9, 9, scales.shape))
        at = slice(c // 128 * 128, c // 128 * 128 + 128)
        part = [f8.decode(t[0][:, at], t[1][:, c // 128:c // 128 + 1], high) for t, high in ((a, 1), (w, 128))]
        want = torch.from_numpy(part[0] @ part[1].T).bfloat16().double().numpy()
        assert np.array_equal(product(a, w, k, "bf16"), want), c


@pytest.mark.parametrize("m,n,k", TILES)
def test_bf16_products_do_not_depend_on_the_run(m, n, k):
    say(f"bf16 product {m}x{n}x{k} twice")
    rng = np.random.default_rng(m + k)
    a, w = packed(rng, m, k), packed(rng, n, k, 128)
    assert np.array_equal(product(a, w, k, "bf16"), product(a, w, k, "bf16"))


# the expert passes' tiles: 256 and 128 rows of the fused pass, 256 x 256, 128 x 256 and 128 x 128 of the down pass
EXPERT_TILES = [("gate_up", 700, 8, 2, 384, 2048), ("gate_up", 900, 8, 1, 256, 2048), ("down", 700, 8, 2, 4096, 384),
                ("down", 900, 8, 1, 2816, 1152), ("down", 900, 8, 1, 2816, 256)]


@pytest.mark.parametrize("part,n,E,k,H,I,kind", [(*tile, kind) for tile in EXPERT_TILES for kind in ("bf16", "fp32", "e4m3")
                                                 if kind != "e4m3" or tile[0] == "gate_up"])
def test_nan_reaches_its_own_outputs_of_an_expert_pass_only(part, n, E, k, H, I, kind):
    say(f"expert tiles {part} n={n} H={H} I={I} {kind} with NaN, and twice")
    ex = Experts(n + H, n, E, k, H, I, holes=0.1)
    get = lambda: ex.run(part, kind)
    decoded = lambda got: f8.decode(*got) if kind == "e4m3" else got
    first, again = get(), get()
    if kind == "e4m3":
        same(first, again)
    else:
        assert np.array_equal(first, again)
    before = decoded(first)
    owner = ex.idx.reshape(-1)
    matrix = "up" if part == "gate_up" else "down"
    act, rows, width = (ex.x, I, I) if part == "gate_up" else (ex.h, H, H)
    a_row = 5
    act[0][a_row, 3] = 0x7f                                  # a code of the activations
    act[1][a_row + 20, -1] = np.nan                          # and a scale
    codes, scales = ex.dev[matrix]
    codes[2 * rows + 130, 1] = 0xff                          # expert 2: a code of row 130
    scales[(3 * rows) // 128 + 1, 0] = float("nan")          # expert 3: a scale of rows 128 .. 255
    after = decoded(get())
    div = k if part == "gate_up" else 1
    hit = np.zeros((n * k, width), bool)
    for r in (a_row, a_row + 20):
        hit[r * div:(r + 1) * div] = True
    hit[owner == 2, 130] = True
    hit[owner == 3, 128:256] = True
    if kind == "e4m3":                                       # a NaN takes its block along
        hit = hit.reshape(n * k, -1, 128).any(2).repeat(128, axis=1)
    hit[owner < 0] = False                                   # in no bin: left as they were
    assert np.all(np.isnan(after[hit]))
    assert np.array_equal(after[~hit], before[~hit], equal_nan=True)
    assert np.all(np.isfinite(before[owner >= 0]))
    ex.close()


# ---- norm, scales of powers of two ---------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 129), (5, 4096), (3, 8200), (2, 20001), (2, 40000)])
def test_norm_into_scales_of_powers_of_two(rows, cols, kind):
    import torch
    say(f"norm {rows}x{cols} {kind} by the power-of-two rule")
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-6, 6, (rows, 1), generator=g).float()))
    x, res = x.to(dtype_of(kind)).cuda(), torch.randn(rows, cols, generator=g).to(dtype_of(kind)).cuda()
    w = (1 + 0.2 * torch.randn(cols, generator=g)).cuda()
    codes, scales, total, _ = norm(x, kind, res, w, "fp32", 1e-6, "pow2")
    h = (x.cpu().double() + res.cpu().double()).to(x.dtype).double().numpy()
    assert np.array_equal(total, h)
    y = f8.rms_norm(h, w.cpu().double().numpy(), 1e-6)
    lim = norm_bound(cols) * np.abs(y)
    for b in range(scales.shape[1]):          # the power of two of a largest magnitude within its bound
        at = slice(128 * b, 128 * (b + 1))
        for r in range(rows):
            top = np.abs(y[r, at])
            ends = [f8.scale_of(v, "pow2") for v in ((top - lim[r, at]).max(), (top + lim[r, at]).max())]
            assert float(scales[r, b]) in ends, (r, b)
    s = spread(scales, rows, cols)
    got = f8.TABLE[codes[:, :cols]] * s
    within(got, y, lim + np.maximum(2.0 ** -4 * (np.abs(y) + lim), s * 2.0 ** -10))
    assert not codes[:, cols:].any()


@pytest.mark.parametrize("cols", [300, 40000])
def test_norm_with_the_largest_eps(cols):
    # the mean and eps together are past fp32's range
    import torch
    say(f"norm of {cols} columns with the largest eps")
    x = (torch.rand(3, cols, generator=torch.Generator().manual_seed(6)) - 0.5).cuda() * (2.0 ** 63 / cols ** 0.5)
    check_norm(x, "fp32", None, torch.ones(cols, device="cuda:0"), "fp32", float(np.finfo(np.float32).max))
