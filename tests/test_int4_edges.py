"""Weights of 4-bit integers at the ends of their ranges: scales that round past fp32, values on the grid.

References and tolerances are test_int4.py's."""
import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as lf
from parity import log
from test_int4 import f64, rounded, short, stored, values


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 128, 256])
def test_pack_scales_that_round_past_the_range(group):
    # 0x7F7FFF80 is half-way between the largest scale, 0x7F7FFF00, and 2^128: the tie goes up, to an infinity
    bits = np.array([0x7F7FFFFF, 0x7F7FFF80, 0x7F7FFF7F, 0x7F7FFF00, 0x7F800000, 0x7FC00001, 0x7F800001, 0x7FFFFFFF], np.uint32)
    bits = np.concatenate([bits, bits | 0x80000000])
    n, k = bits.size, 264
    G = -(-k // group)
    s = np.tile(bits, (G, 1))
    q = np.tile(np.arange(k, dtype=np.uint8)[:, None] % 16, (1, n))
    z = np.tile(np.arange(n, dtype=np.uint8)[None], (G, 1))
    log(f"pack scales past the range, group {group}")
    got = lf.lora_int4_pack(torch.from_numpy(q).cuda(), torch.from_numpy(s.view(np.float32)).cuda(), torch.from_numpy(z).cuda(), group=group)
    largest = float(np.uint32(0x7F7FFF00).view(np.float32))
    held = np.where(np.isin(s & 0x7FFFFFFF, (0x7F7FFF7F, 0x7F7FFF00)), np.where(s >> 31, -largest, largest), np.nan)
    want = stored(q, held, z, group)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    back, W = f64(lf.lora_int4_dequantize(got)), values(q, held, z, group)
    nan = np.isnan(W)
    assert nan.any() and not nan.all() and np.array_equal(np.isnan(back), nan)
    assert np.array_equal(back[~nan], rounded(W)[~nan])  # (an overflowing value is an infinity in both)
