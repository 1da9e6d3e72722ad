"""e4m3 on the GPU at the edges of its range: sizes past one launch, and what the 8-bit matrix instructions make of NaN,
extreme scales and single inputs."""
import numpy as np
import pytest

import trellis_quantized_moe_expert_amd as q
from f8_util import RULE, TYPE
from gpu_util import say
from oracle import f8

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
