"""Weights of 4-bit integers at the ends of their ranges: scales that round past fp32, values on the grid.

References and tolerances are test_int4.py's."""
import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as lf
from parity import log
from test_int4 import f64, ref_quantize, rounded, short, stored, values


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


def on_the_grid(k, n, group, symmetric, seed):
    """(W (k x n) of exact values s (q - z), q, s, z), each group with both ends of the codes it can have."""
    rng = np.random.default_rng(seed)
    G = -(-k // group)
    # s of four significant bits: with four of q - z every value is a bf16
    s = rng.integers(8, 16, (G, n)) * 2.0 ** rng.integers(-12, 4, (G, n))
    z = np.full((G, n), 8) if symmetric else rng.integers(0, 16, (G, n))
    q = rng.integers(1 if symmetric else 0, 16, (k, n))
    for b in range(G):
        q[b * group], q[min(b * group + 5, k - 1)] = (1, 15) if symmetric else (0, 15)
    W = values(q, s, z, group)
    assert np.array_equal(rounded(W), W) and np.array_equal(short(s), s)
    return torch.from_numpy(W).bfloat16(), q.astype(np.uint8), s, z


GRID = [(192, 24, 32, False), (192, 24, 64, True), (264, 40, 128, False), (392, 24, 128, True), (520, 16, 256, False), (904, 24, 384, True)]


@pytest.mark.parametrize("k,n,group,symmetric", GRID)
def test_definition_keeps_values_on_the_grid(k, n, group, symmetric):
    W, q, s, z = on_the_grid(k, n, group, symmetric, k)
    q2, s2, z2 = ref_quantize(f64(W), group, symmetric)
    assert np.array_equal(q2, q) and np.array_equal(s2, s) and np.array_equal(z2, z)
    assert np.array_equal(values(q2, s2, z2, group), f64(W))


@pytest.mark.gpu
@pytest.mark.parametrize("k,n,group,symmetric", GRID)
def test_quantize_keeps_values_on_the_grid(k, n, group, symmetric):
    W, q, s, z = on_the_grid(k, n, group, symmetric, k + 1)
    log(f"grid {k} x {n} group {group}")
    got, want = lf.lora_int4_quantize(W.cuda(), group, symmetric=symmetric), stored(q, s, z, group)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    assert torch.equal(lf.lora_int4_dequantize(got).cpu(), W)
    again = lf.lora_int4_quantize(lf.lora_int4_dequantize(got), group, symmetric=symmetric)
    assert torch.equal(again.codes, got.codes) and torch.equal(again.scales, got.scales)
