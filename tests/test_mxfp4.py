"""Frozen weights in MXFP4: packing, and the layers over them.

The reference is written here from the format's definition, in 64 bits with
numpy; it shares nothing with the library.

Tolerances, derived:
* packing and unpacking are exact: codes and scales follow from W alone, and
  every value is a bf16.
* a product's entry is an fp32 sum of k exact products (bf16 times bf16 fits
  fp32) rounded once to bf16, so it is off by at most half a bf16 step, 2^-8 of
  its value, and k 2^-24 of the sum of its terms' magnitudes (every addition
  rounds by half an fp32 step, 2^-24, of a partial sum no larger than that).
* the LoRA term adds the same for S (k terms) carried through alpha S B (r
  terms), and the split of alpha S into two bf16, which keeps it to 2^-16.
  fp32 dS in the backward likewise.
"""
import os

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as lf
import oracle
from lora_fine_tuning_amd import _lib
from parity import bf16_randn, log, offset_view

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BF, HALF = 2.0 ** -8, 2.0 ** -24
FAKE = 0x10000  # aligned, never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


# ---- the format, from its definition ---------------------------------------------------------

def ref_pack(W):
    """(codes (k, n) 0..15, scale bytes (ceil(k/32), n)) of a float64 matrix of bf16 values."""
    k, n = W.shape
    codes, scales = np.zeros((k, n), np.uint8), np.zeros((-(-k // 32), n), np.uint8)
    for b in range(scales.shape[0]):
        blk = W[32 * b:32 * b + 32]
        bad = ~np.isfinite(blk).all(0)
        w = np.where(np.isfinite(blk), blk, 0.0)
        top = np.abs(w).max(0)
        e = np.zeros(n, int)
        some = top > 0
        e[some] = np.floor(np.log2(top[some])).astype(int) - 2
        e[some] += top[some] / 2.0 ** e[some] >= 7
        e = np.where(some, np.clip(e, -125, 125), 0)
        y = np.abs(w) / 2.0 ** e
        d = np.abs(y[..., None] - GRID)
        # nearest; of two equally near ones the even index
        near = d == d.min(-1, keepdims=True)
        even = near & (np.arange(8) % 2 == 0)
        c = np.where(even.any(-1), even.argmax(-1), near.argmax(-1)).astype(np.uint8)
        c[:, bad] = 0
        codes[32 * b:32 * b + 32] = c + 8 * (np.signbit(blk) & ~bad)
        scales[b] = np.where(bad, 255, e + 127)
    return codes, scales


def ref_values(codes, scales):
    v = np.where(codes >= 8, -1.0, 1.0) * GRID[codes & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(float) - 127))
    return v * np.repeat(s, 32, 0)[:codes.shape[0]]


def unpacked(W4):
    """(codes (KB * 32, N16 * 16), scales (KB, N16 * 16)) from the stored layout."""
    c, s = W4.codes.cpu().numpy(), W4.scales.cpu().numpy()
    n16, kb = s.shape[:2]
    codes = np.zeros((kb * 32, n16 * 16), np.uint8)
    scales = np.zeros((kb, n16 * 16), np.uint8)
    for g in range(n16):
        for j in range(16):
            scales[:, 16 * g + j] = s[g, :, j]
            codes[0::2, 16 * g + j] = (c[g, :, j] & 15).reshape(-1)
            codes[1::2, 16 * g + j] = (c[g, :, j] >> 4).reshape(-1)
    return codes, scales


def packed(codes, scales, k, n, device="cuda"):
    """An Mxfp4Weight from plain (k, n) codes and (blocks, n) scales."""
    n16, kb = -(-n // 16), 4 * -(-k // 128)
    c = np.zeros((kb * 32, n16 * 16), np.uint8)
    c[:k, :n] = codes
    s = np.full((kb, n16 * 16), 127, np.uint8)
    s[:scales.shape[0], :n] = scales
    by = (c[0::2] | c[1::2] << 4).reshape(kb, 16, n16, 16).transpose(2, 0, 3, 1)
    return lf.Mxfp4Weight(torch.from_numpy(np.ascontiguousarray(by)).to(device),
                          torch.from_numpy(np.ascontiguousarray(s.reshape(kb, n16, 16).transpose(1, 0, 2))).to(device),
                          k, n)


def test_reference_round_trip_and_error_bound():
    # the definition itself: over the scale the largest value t lies in [3.5, 7), and a value y <= t is off
    # by at most 1/2 up to 4 (1/7 of t), by y - 4 <= t - 4 up to 5 and by 1 from 5 on (1/5 of t); and a
    # value on the grid is exact
    rng = np.random.default_rng(0)
    W = f64(torch.from_numpy(rng.standard_normal((96, 24))).bfloat16())
    c, s = ref_pack(W)
    V = ref_values(c, s)
    top = np.repeat(np.abs(W).reshape(3, 32, 24).max(1), 32, 0)
    assert (np.abs(V - W) <= top / 5 + 1e-12).all()
    c2, s2 = ref_pack(V)
    assert np.array_equal(ref_values(c2, s2), V)


# ---- refusals (host) ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("host-only checks; a GPU is visible")
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    return _lib.load()


def test_sizes():
    lib = _lib.load()
    for k, n, want in ((8, 8, 4 * 256), (128, 16, 4 * 256), (136, 16, 8 * 256), (4096, 14336, 128 * 896 * 256)):
        assert lib.lora_mxfp4_codes_size(k, n) == want
        assert lib.lora_mxfp4_scales_size(k, n) == want // 16
    assert lib.lora_mxfp4_codes_size(0, 8) == 0 and lib.lora_mxfp4_codes_size(8, -1) == 0
    # without rows the weight is not read: the bf16 layer's scratch alone
    assert lf.lora_mxfp4_linear_bwd_workspace_size(0, 64, 64, 8) == _lib.lora_linear_bwd_workspace_size(0, 64, 64, 8)
    assert lf.lora_mxfp4_linear_bwd_workspace_size(8192, 64, 64, 8) > 0
    assert lf.lora_mxfp4_frozen_fwd_workspace_size(0, 64, 64) == 0
    assert lf.lora_mxfp4_frozen_fwd_workspace_size(-1, 64, 64) == 0


def test_pack_rejects(lib):
    for f in (lib.lora_mxfp4_quantize, lib.lora_mxfp4_dequantize):
        assert f(None, 64, 64, FAKE, FAKE, None) == INVALID
        if f is lib.lora_mxfp4_quantize:
            assert f(FAKE, 60, 64, FAKE, FAKE, None) == INVALID       # k % 8
            assert f(FAKE, 64, 20, FAKE, FAKE, None) == INVALID       # n % 8
            assert f(FAKE, 0, 64, FAKE, FAKE, None) == INVALID
            assert f(FAKE + 8, 64, 64, FAKE, FAKE, None) == INVALID
            assert f(FAKE, 64, 64, FAKE + 8, FAKE, None) == INVALID
            assert f(FAKE, 64, 64, FAKE, FAKE + 8, None) == INVALID
            assert f(FAKE, 64, 64, FAKE, None, None) == INVALID
            assert f(FAKE, 1 << 30, 1 << 30, FAKE, FAKE, None) == INVALID  # too large
    assert lib.lora_mxfp4_dequantize(FAKE, FAKE, 60, 64, FAKE, None) == INVALID
    assert lib.lora_mxfp4_dequantize(FAKE, FAKE, 64, 64, FAKE + 2, None) == INVALID


def test_layer_rejects(lib):
    F, big = FAKE, 1 << 40
    fz = lib.lora_mxfp4_frozen_fwd
    assert fz(F, F, F, 4, 60, 64, F, F, big, None) == INVALID
    assert fz(F, F, F, -1, 64, 64, F, F, big, None) == INVALID
    assert fz(None, F, F, 4, 64, 64, F, F, big, None) == INVALID
    assert fz(F + 8, F, F, 4, 64, 64, F, F, big, None) == INVALID
    assert fz(F, F, F + 4, 4, 64, 64, F, F, big, None) == INVALID
    assert fz(None, F, F, 0, 64, 64, None, None, 0, None) == 0
    assert lib.lora_mxfp4_frozen_bwd(F, F, F, 4, 64, 64, None, F, big, None) == INVALID
    need = lib.lora_mxfp4_frozen_bwd_workspace_size(4096, 4096, 4096)
    if need:
        assert lib.lora_mxfp4_frozen_bwd(F, F, F, 4096, 4096, 4096, F, F, need - 1, None) == WORKSPACE

    def fwd(**kw):
        a = dict(X=F, c=F, s=F, A=F, B=F, m=64, k=64, n=64, r=8, p=0.1, off=0, Y=F, S=F, keep=F, ws=F, wsb=big)
        a.update(kw)
        return lib.lora_mxfp4_linear_fwd(a["X"], a["c"], a["s"], a["A"], a["B"], a["m"], a["k"], a["n"], a["r"], 1.0,
                                         a["p"], 0, a["off"], a["Y"], a["S"], a["keep"], a["ws"], a["wsb"], None)

    for kw in (dict(X=None), dict(c=None), dict(c=F + 8), dict(s=None), dict(A=None), dict(B=None), dict(Y=None),
               dict(S=None), dict(r=0), dict(r=257), dict(p=1.0), dict(p=-0.1), dict(off=4), dict(keep=None),
               dict(k=12), dict(n=12), dict(S=F + 2), dict(keep=F + 2), dict(p=float("nan"))):
        assert fwd(**kw) == INVALID, kw
    need = lib.lora_mxfp4_linear_fwd_workspace_size(512, 4096, 4096, 256)  # partial sums of S at least
    assert need > 0 and fwd(m=512, k=4096, n=4096, r=256, wsb=need - 1) == WORKSPACE
    assert fwd(r=256, n=1 << 22) == UNSUPPORTED
    assert fwd(m=0, X=None, Y=None, S=None, keep=None, ws=None, wsb=0) == 0

    def bwd(**kw):
        a = dict(dY=F, X=F, c=F, s=F, A=F, B=F, S=F, keep=F, m=64, k=64, n=64, r=8, p=0.1, dX=F, dA=F, dB=F, ws=F,
                 wsb=big)
        a.update(kw)
        return lib.lora_mxfp4_linear_bwd(a["dY"], a["X"], a["c"], a["s"], a["A"], a["B"], a["S"], a["keep"], a["m"],
                                         a["k"], a["n"], a["r"], 1.0, a["p"], a["dX"], a["dA"], a["dB"], a["ws"],
                                         a["wsb"], None)

    for kw in (dict(dY=None), dict(X=None), dict(c=None), dict(s=F + 1), dict(dA=None), dict(dB=None), dict(S=None),
               dict(keep=None), dict(r=300), dict(p=1.5), dict(dX=F + 2), dict(k=20), dict(ws=None)):
        assert bwd(**kw) == INVALID, kw
    assert bwd(wsb=0) == WORKSPACE and bwd(dX=None, wsb=0) == WORKSPACE
    assert bwd(r=256, k=1 << 22) == UNSUPPORTED

    mf, mb = lib.multi_lora_mxfp4_linear_fwd, lib.multi_lora_mxfp4_linear_bwd
    assert mf(F, F, F, F, 0, F, F, 1, 64, 64, 64, 16, 0, 0, F, F, F, F, big, None) == INVALID
    assert mf(F, F, F, F, 2, F, F, 0, 64, 64, 64, 16, 0, 0, F, F, F, F, big, None) == INVALID
    assert mf(F, F, F, F, 2, F, F, 1, 64, 64, 64, 16, 0, 0, F, F, None, F, big, None) == INVALID
    assert mf(F, F, F, F, 2, F, F, 1, 64, 64, 64, 16, 0, 4, F, F, F, F, big, None) == INVALID
    assert mf(F, F, F, F, 2, F, F, 1, 64, 64, 64, 16, 0, 0, F, F, F, F, 0, None) == WORKSPACE
    assert mb(F, F, F, F, F, 2, F, F, 1, F, F, 64, 64, 64, 300, F, F, big, None) == INVALID
    assert mb(F, F, F, F, F, 2, F, F, 1, F, None, 64, 64, 64, 16, F, F, big, None) == INVALID
    assert mb(F, F, F, F, F, 2, F, F, 1, F, F, 64, 64, 64, 16, F, F, 0, None) == WORKSPACE


def test_binding_rejects():
    # everything but the device is checked on CPU tensors too
    W = lf.Mxfp4Weight(torch.zeros(4, 4, 16, 16, dtype=torch.uint8), torch.zeros(4, 4, 16, dtype=torch.uint8), 64, 64)
    X = torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="Mxfp4Weight"):
        lf.lora_mxfp4_frozen_fwd(X, X)
    with pytest.raises(TypeError, match="uint8"):
        lf.lora_mxfp4_frozen_fwd(X, W._replace(codes=W.codes.int()))
    with pytest.raises(ValueError, match="device"):
        lf.lora_mxfp4_frozen_fwd(X, W)
    with pytest.raises(TypeError, match="bfloat16"):
        lf.lora_mxfp4_quantize(X.float())


# ---- packing (GPU) --------------------------------------------------------------------------------

def special_weight():
    """Every tie, zeros of both signs, subnormals, the largest values, lone values beside huge ones."""
    k, n = 96, 40
    g = torch.Generator().manual_seed(1)
    W = bf16_randn((k, n), 1.0, g)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0])
    W[:32, 0] = torch.cat([ties, -ties]).bfloat16()            # top 6: scale 1
    W[:32, 1] = W[:32, 0] * 2.0 ** -20
    W[:32, 2] = 0.0
    W[:32, 3] = -0.0
    W[:32, 4] = 2.0 ** -133                                    # the smallest subnormal
    W[:32, 5] = 3.3895313892515355e38                          # the largest bf16
    W[:32, 6] = 0.0
    W[5, 6] = -3.3895313892515355e38
    W[:32, 7] = 6.96875                                        # just below the next scale
    W[:32, 8] = 7.0                                            # at it
    W[:32, 9] = torch.linspace(-7, 7, 32).bfloat16()
    W[:32, 10] = 2.0 ** -126
    W[:32, 11] = torch.tensor([2.0 ** -e for e in range(32)]).bfloat16()
    return W


PACK_SHAPES = [(8, 8), (32, 16), (40, 24), (128, 256), (136, 8), (1000, 1032), (264, 520), (2048, 4104)]


@pytest.mark.gpu
@pytest.mark.parametrize("k,n", PACK_SHAPES)
def test_pack_matches_definition(k, n):
    log(f"pack {k} x {n}")
    W = bf16_randn((k, n), k ** -0.5, torch.Generator().manual_seed(k + n))
    check_pack(W)


def check_pack(W):
    k, n = W.shape
    W4 = lf.lora_mxfp4_quantize(W.cuda())
    back = lf.lora_mxfp4_dequantize(W4)
    torch.cuda.synchronize()
    codes, scales = ref_pack(f64(W))
    got_c, got_s = unpacked(W4)
    nb = scales.shape[0]
    assert np.array_equal(got_s[:nb, :n], scales)
    # codes 0 and 8 are both zero
    same = (got_c[:k, :n] == codes) | ((got_c[:k, :n] & 7) + (codes & 7) == 0)
    assert same.all(), np.argwhere(~same)[:4]
    assert not got_c[k:].any() and not got_c[:, n:].any()          # padding holds zero codes
    assert (got_s[nb:] == 127).all() and (got_s[:, n:] == 127).all()
    np.testing.assert_array_equal(f64(back), ref_values(codes, scales))


@pytest.mark.gpu
def test_pack_special_values():
    check_pack(special_weight())


@pytest.mark.gpu
def test_pack_every_bf16():
    # each finite bf16 with 30 neighbours and a power of two that sets the block's scale
    bits = np.arange(1 << 15, dtype=np.uint16)
    vals = torch.from_numpy(bits.astype(np.int16)).view(torch.bfloat16)
    vals = vals[torch.isfinite(vals)]
    n = 1056
    cols = torch.zeros(31 * n, dtype=torch.bfloat16)
    cols[:vals.numel()] = vals
    cols = cols.view(n, 31).t()
    top = torch.ceil(torch.log2(cols.double().amax(0).clamp_min(2.0 ** -133)))
    for shift in (0, 1, 2, 3):
        lead = (2.0 ** (top + shift).clamp_max(127)).bfloat16()[None]
        check_pack(torch.cat([cols, lead]).contiguous())
        check_pack(torch.cat([-lead, -cols]).contiguous())


@pytest.mark.gpu
def test_pack_marks_blocks_with_infinities_and_nans():
    W = bf16_randn((72, 24), 1.0, torch.Generator().manual_seed(3))
    W[3, 1], W[40, 5], W[71, 7] = float("inf"), float("nan"), -float("inf")
    check_pack(W)
    W4 = lf.lora_mxfp4_quantize(W.cuda())
    back = lf.lora_mxfp4_dequantize(W4).cpu()
    bad = torch.zeros(72, 24, dtype=torch.bool)
    bad[:32, 1] = bad[32:64, 5] = bad[64:, 7] = True
    assert torch.equal(torch.isnan(back), bad)
    # a product over it is NaN where such a column takes part, and nowhere else
    X = bf16_randn((5, 72), 1.0, torch.Generator().manual_seed(4)).cuda()
    Y = lf.lora_mxfp4_frozen_fwd(X, W4).cpu()
    assert torch.equal(torch.isnan(Y).all(0), bad.any(0)) and torch.equal(torch.isnan(Y).any(0), bad.any(0))
    dX = lf.lora_mxfp4_frozen_bwd(bf16_randn((5, 24), 1.0, torch.Generator().manual_seed(5)).cuda(), W4).cpu()
    assert torch.equal(torch.isnan(dX).any(0), bad.any(1))


@pytest.mark.gpu
def test_every_scale_byte_reads_as_its_power():
    k, n = 32, 256
    codes = np.tile(np.arange(16, dtype=np.uint8)[:, None], (2, n))
    scales = np.arange(256, dtype=np.uint8)[None]
    back = lf.lora_mxfp4_dequantize(packed(codes, scales, k, n)).cpu()
    want = torch.from_numpy(ref_values(codes, scales)).to(torch.bfloat16)  # to nearest even, past the range inf
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(back[ok], want[ok])


# ---- the layers (GPU) -------------------------------------------------------------------------------

def layer_case(m, k, n, r, seed):
    g = torch.Generator().manual_seed(seed)
    X = bf16_randn((m, k), 1.0, g)
    W4 = lf.lora_mxfp4_quantize(bf16_randn((k, n), k ** -0.5, g).cuda())
    A = bf16_randn((k, r), k ** -0.5, g)
    B = bf16_randn((r, n), 0.02 ** 0.5, g)
    dY = bf16_randn((m, n), 1.0, g)
    codes, scales = unpacked(W4)
    W = ref_values(codes[:k, :n], scales[:-(-k // 32), :n])
    return X, W4, W, A, B, dY


def near(name, got, want, slack):
    """Every entry within half a bf16 step of `want` and `slack` (an array) of the sums before it."""
    got = f64(got)
    assert np.isfinite(got).all(), name
    bound = BF * np.abs(want) + (1 + BF) * slack
    over = np.abs(got - want) - bound
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[at] <= 0, f"{name}{at}: {got[at]!r}, want {want[at]!r} within {bound[at]:.3g}"


# single tokens, every count of 16-row tiles and their edges, k and n that end inside blocks and groups
FROZEN = [(1, 8, 8), (1, 128, 16), (2, 40, 24), (1, 4096, 264), (3, 1032, 520), (7, 136, 8), (15, 264, 136),
          (16, 520, 1032), (17, 392, 72), (31, 2056, 104), (33, 640, 200), (48, 1000, 312), (64, 4104, 96), (65, 256, 264),
          (100, 904, 136), (127, 72, 528), (128, 1280, 256), (129, 136, 264), (200, 2064, 120), (257, 520, 520),
          (300, 3000, 264), (513, 264, 1032), (1030, 400, 776), (2050, 136, 136)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n", FROZEN)
def test_frozen_forward_and_backward(m, k, n):
    log(f"frozen m={m} k={k} n={n}")
    X, W4, W, _, _, dY = layer_case(m, k, n, 8, seed=m + k + n)
    Yb = torch.full((m + 3, n), 5.0, dtype=torch.bfloat16, device="cuda")  # rows behind the last stay as they were
    dXb = torch.full((m + 3, k), 5.0, dtype=torch.bfloat16, device="cuda")
    lf.lora_mxfp4_frozen_fwd(X.cuda(), W4, Y=Yb[:m])
    lf.lora_mxfp4_frozen_bwd(dY.cuda(), W4, dX=dXb[:m])
    torch.cuda.synchronize()
    assert (Yb[m:] == 5).all() and (dXb[m:] == 5).all()
    x, dy = f64(X), f64(dY)
    near("Y", Yb[:m], x @ W, k * HALF * (np.abs(x) @ np.abs(W)))
    near("dX", dXb[:m], dy @ W.T, n * HALF * (np.abs(dy) @ np.abs(W).T))


# sums split over many work-groups, and every number of row tiles, in both directions
DEEP = [(1, 4096, 4104), (9, 1288, 8200), (24, 4096, 2048), (70, 2568, 4096), (128, 1024, 6152), (400, 776, 2056), (1100, 1288, 1032),
        (999, 4104, 2056), (1500, 2056, 1032), (1900, 1800, 776)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n", DEEP)
def test_frozen_deep(m, k, n):
    test_frozen_forward_and_backward(m, k, n)


LAYER = [
    # m, k, n, r, alpha, p
    (1, 4096, 520, 16, 2.0, 0.0), (1, 264, 136, 5, -0.7, 0.0), (1, 72, 40, 1, 2.0, 0.3), (2, 1032, 264, 64, 0.5, 0.0),
    (5, 2056, 136, 200, 1.0, 0.0), (16, 520, 1032, 8, 2.0, 0.1), (17, 136, 72, 33, 1.0, 0.0), (40, 1288, 264, 128, 0.5, 0.0),
    (48, 392, 520, 256, 1.0, 0.05), (63, 264, 264, 13, 2.0, 0.0), (100, 904, 392, 32, 2.0, 0.2), (130, 648, 520, 100, 1.0, 0.0),
    (333, 1032, 776, 5, 2.0, 0.2), (520, 400, 264, 130, 0.5, 0.1), (700, 264, 1032, 16, 2.0, 0.1),
    # S formed beside the product over several row tiles, at odd ranks
    (65, 1032, 264, 7, 1.0, 0.0), (100, 4104, 136, 31, -2.0, 0.0), (128, 2056, 520, 66, 0.5, 0.0), (128, 264, 72, 255, 1.0, 0.0),
    # more rows, and a contraction split over work-groups in both directions
    (1030, 520, 136, 16, 2.0, 0.0), (2, 8200, 4104, 16, 2.0, 0.1), (30, 4104, 8200, 12, 2.0, 0.0),
    (1400, 2056, 1288, 40, 2.0, 0.1),
]


def layer_reference(X, W, A, B, dY, alpha, p, seed, offset):
    """(outputs, slacks) of the layer in 64 bits."""
    x, a, b, dy = f64(X), f64(A), f64(B), f64(dY)
    m, k = x.shape
    n, r = W.shape[1], a.shape[1]
    p32 = float(np.float32(p))
    keep = oracle.keep_mask(seed, offset, range(m), k, np.float32(p)) if p > 0 else np.ones((m, k))
    xd = x * keep / (1 - p32)
    S, dS = xd @ a, alpha * (dy @ b.T)
    ab = np.abs
    eS = (k + 2) * HALF * (ab(xd) @ ab(a))
    edS = (n + 2) * HALF * abs(alpha) * (ab(dy) @ ab(b).T)
    split = 2.0 ** -16
    out = {"S": S, "Y": x @ W + alpha * (S @ b), "dX": dy @ W.T + keep / (1 - p32) * (dS @ a.T), "dA": xd.T @ dS,
           "dB": alpha * (S.T @ dy)}
    up = abs(alpha) * (ab(S) @ ab(b))
    down = (ab(dS) @ ab(a).T) / (1 - p32)
    slack = {
        "S": eS,
        "Y": (k + r + 4) * HALF * (ab(x) @ ab(W) + up) + split * up + abs(alpha) * (eS @ ab(b)),
        "dX": (n + r + 4) * HALF * (ab(dy) @ ab(W).T + down) + split * down + (edS @ ab(a).T) / (1 - p32),
        "dA": (m + 4) * HALF * (ab(xd).T @ ab(dS)) + split * (ab(xd).T @ ab(dS)) + ab(xd).T @ edS,
        "dB": abs(alpha) * ((m + 4) * HALF * (ab(S).T @ ab(dy)) + split * (ab(S).T @ ab(dy)) + eS.T @ ab(dy)),
    }
    return out, slack


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(LAYER)))
def test_layer_forward_and_backward(case):
    m, k, n, r, alpha, p = LAYER[case]
    log(f"layer m={m} k={k} n={n} r={r} p={p}")
    X, W4, W, A, B, dY = layer_case(m, k, n, r, seed=900 + case)
    Xd, Ad, Bd = X.cuda(), A.cuda(), B.cuda()
    Y, S, keep = lf.lora_mxfp4_linear_fwd(Xd, W4, Ad, Bd, alpha, p, 7, 16)
    dX, dA, dB = lf.lora_mxfp4_linear_bwd(dY.cuda(), Xd, W4, Ad, Bd, S, keep, alpha, p)
    torch.cuda.synchronize()
    if p > 0:
        assert torch.equal(keep, lf.lora_dropout_mask(7, 16, m, k, p))
    want, slack = layer_reference(X, W, A, B, dY, alpha, p, 7, 16)
    got_s = f64(S)
    assert (np.abs(got_s - want["S"]) <= slack["S"] + 1e-30).all()
    for name, t in (("Y", Y), ("dX", dX), ("dA", dA), ("dB", dB)):
        near(name, t, want[name], slack[name])
    # without an input gradient the others stay the same
    none, dA2, dB2 = lf.lora_mxfp4_linear_bwd(dY.cuda(), Xd, W4, Ad, Bd, S, keep, alpha, p, want_dX=False)
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,r", [(1, 136, 8), (40, 1080, 40), (130, 2056, 72), (700, 264, 16)])
def test_mask_is_written_whole(m, k, r):
    # every word of the mask, its bits past k among them, whatever the buffer held; p = 0 keeps everything, and
    # a p whose threshold is zero drops nothing
    n = 264
    X, W4, W, A, B, dY = layer_case(m, k, n, r, seed=37)
    for p in (0.0, 2.0 ** -20, 0.3, 0.9999):
        keep = torch.full((m + 1, (k + 31) // 32), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
        Y, S, got = lf.lora_mxfp4_linear_fwd(X.cuda(), W4, A.cuda(), B.cuda(), 2.0, p, 11, 24, keep_bits=keep[:m])
        torch.cuda.synchronize()
        assert got.data_ptr() == keep.data_ptr() and (keep[m] == 0x5A5A5A5A).all()
        assert torch.equal(got, lf.lora_dropout_mask(11, 24, m, k, p))
        want, slack = layer_reference(X, W, A, B, dY, 2.0, p, 11, 24)
        near("Y", Y, want["Y"], slack["Y"])


@pytest.mark.gpu
@pytest.mark.parametrize("m,r,p", [(1, 16, 0.0), (33, 9, 0.0), (33, 64, 0.1), (300, 40, 0.1), (700, 16, 0.0)])
def test_unaligned_adapter_gives_the_same(m, r, p):
    # A and B one element past a 16-byte boundary: the same sums in the same order
    k, n = 1032, 520
    X, W4, W, A, B, dY = layer_case(m, k, n, r, seed=31)
    X, dY = X.cuda(), dY.cuda()

    def run(A, B):
        Y, S, keep = lf.lora_mxfp4_linear_fwd(X, W4, A, B, 2.0, p, 3, 0)
        return (Y, S, *lf.lora_mxfp4_linear_bwd(dY, X, W4, A, B, S, keep, 2.0, p))

    Y, S, dX, dA, dB = run(offset_view(A), offset_view(B))
    want, slack = layer_reference(X.cpu(), W, A, B, dY.cpu(), 2.0, p, 3, 0)
    for name, t in (("Y", Y), ("dX", dX), ("dA", dA), ("dB", dB)):
        near(name, t, want[name], slack[name])
    assert (np.abs(f64(S) - want["S"]) <= slack["S"] + 1e-30).all()


@pytest.mark.gpu
def test_gradient_against_differences():
    # d/dX, d/dA, d/dB of <Y, dY>: the layer is linear in each of the three, so a difference of two
    # forwards is exact up to rounding; steps are whole bf16 values
    m, k, n, r = 24, 136, 72, 8
    X, W4, W, A, B, dY = layer_case(m, k, n, r, seed=41)
    Xd, Ad, Bd, dYd = X.cuda(), A.cuda(), B.cuda(), dY.cuda()
    _, S, keep = lf.lora_mxfp4_linear_fwd(Xd, W4, Ad, Bd, 2.0, 0.2, 3, 0)
    grads = dict(zip("XAB", lf.lora_mxfp4_linear_bwd(dYd, Xd, W4, Ad, Bd, S, keep, 2.0, 0.2)))
    g = torch.Generator().manual_seed(5)
    for name, t in (("X", Xd), ("A", Ad), ("B", Bd)):
        d = torch.sign(torch.randn(t.shape, generator=g)).cuda().bfloat16()
        up, down = ({"X": Xd, "A": Ad, "B": Bd} | {name: v} for v in (d, -d))  # linear: take the two at +-d alone
        other = lambda z: lf.lora_mxfp4_linear_fwd(z["X"], W4, z["A"], z["B"], 2.0, 0.2, 3, 0)[0].double()  # noqa: E731
        Yu, Yd = other(up), other(down)
        diff = ((Yu - Yd) * dYd.double()).sum().item() / 2
        dot = (grads[name].double() * d.double()).sum().item()
        # each Y entry is rounded by 2^-8 of itself, each gradient entry too
        bound = BF * ((Yu.abs() + Yd.abs()) * dYd.double().abs()).sum().item() / 2
        bound += BF * grads[name].double().abs().sum().item()
        assert abs(diff - dot) <= bound, (name, diff, dot, bound)


@pytest.mark.gpu
def test_extreme_activations():
    # zeros, and rows near the end of bf16's range: no overflow where the true result is finite
    m, k, n = 20, 264, 136
    X, W4, W, _, _, _ = layer_case(m, k, n, 8, seed=77)
    X[3] = 0
    X[7] *= 2.0 ** 60
    X[8] *= 2.0 ** -60
    Y = lf.lora_mxfp4_frozen_fwd(X.cuda(), W4)
    near("Y", Y, f64(X) @ W, k * HALF * (np.abs(f64(X)) @ np.abs(W)))
    assert not Y[3].any()
    X[5, 9] = float("inf")
    X[6, 1] = float("nan")
    Y = lf.lora_mxfp4_frozen_fwd(X.cuda(), W4).cpu()
    rows = torch.isfinite(Y).all(1)
    assert rows[[i for i in range(m) if i not in (5, 6)]].all() and torch.isnan(Y[6]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 50, 600])
def test_mixed_matches_definition(m):
    k, n, ranks = 520, 264, [16, 8, 40, 5]
    alphas, ps = [2.0, 1.0, 0.5, -1.0], [0.1, 0.0, 0.2, 0.05]
    seg_off, seg_ad = [0, m // 4, m // 4, m // 2, m], [1, 3, 2, 0]
    g = torch.Generator().manual_seed(m)
    X, W4, W, _, _, dY = layer_case(m, k, n, 8, seed=60 + m)
    As = [bf16_randn((k, r), k ** -0.5, g).cuda() for r in ranks]
    Bs = [bf16_randn((r, n), 0.02 ** 0.5, g).cuda() for r in ranks]
    dAs, dBs = [torch.full_like(a, 7.0) for a in As], [torch.full_like(b, 7.0) for b in Bs]
    table = lf.adapter_table(As, Bs, alphas, ps, dAs, dBs)
    so = torch.tensor(seg_off, dtype=torch.int64, device="cuda")
    sa = torch.tensor(seg_ad, dtype=torch.int32, device="cuda")
    Y, S, keep = lf.multi_lora_mxfp4_linear_fwd(X.cuda(), W4, table, 4, so, sa, 40, 3, 8)
    dX = lf.multi_lora_mxfp4_linear_bwd(dY.cuda(), X.cuda(), W4, table, 4, so, sa, S, keep, 40)
    torch.cuda.synchronize()
    used = set()
    for s, a in enumerate(seg_ad):
        lo, hi = seg_off[s], seg_off[s + 1]
        want, slack = layer_reference(X[lo:hi], W, As[a], Bs[a], dY[lo:hi], alphas[a], ps[a], 3, 8 + lo * k)
        near(f"Y[{s}]", Y[lo:hi], want["Y"], slack["Y"])
        near(f"dX[{s}]", dX[lo:hi], want["dX"], slack["dX"])
        near(f"dA[{a}]", dAs[a], want["dA"], slack["dA"])
        near(f"dB[{a}]", dBs[a], want["dB"], slack["dB"])
        used.add(a)
    assert used == set(range(4))  # (an adapter with no rows gets zeros: its reference is an empty sum)


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n,nseg,r_max", [(1, 136, 72, 1, 8), (16, 4104, 264, 16, 64), (40, 1032, 520, 7, 128), (100, 264, 136, 3, 256),
                                              (128, 2056, 264, 5, 40), (200, 520, 136, 300, 16), (1000, 520, 264, 4, 33)])
def test_mixed_s_and_mask_are_whole(m, k, n, nseg, r_max):
    # S of every row, zeros past its rank, and every bit of the mask
    g = torch.Generator().manual_seed(m + nseg)
    X, W4, W, _, _, dY = layer_case(m, k, n, 8, seed=260 + m)
    ranks = [1 + int(torch.randint(0, r_max, (1,), generator=g)) for _ in range(min(nseg, 6))] + [r_max]
    ps = [(0.0, 0.1, 0.3)[i % 3] for i in range(len(ranks))]
    As = [bf16_randn((k, r), k ** -0.5, g) for r in ranks]
    Bs = [bf16_randn((r, n), 0.02 ** 0.5, g) for r in ranks]
    cuts = torch.randint(0, m + 1, (nseg - 1,), generator=g).sort().values.tolist()
    seg_off = [0, *cuts, m]
    seg_ad = torch.randint(0, len(ranks), (nseg,), generator=g).tolist()
    Ad, Bd = [a.cuda() for a in As], [b.cuda() for b in Bs]  # (a table holds addresses only)
    table = lf.adapter_table(Ad, Bd, [0.5] * len(ranks), ps)
    so = torch.tensor(seg_off, dtype=torch.int64, device="cuda")
    sa = torch.tensor(seg_ad, dtype=torch.int32, device="cuda")
    S = torch.full((m, r_max), float("nan"), device="cuda")
    keep = torch.full((m, (k + 31) // 32), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    Y, S, keep = lf.multi_lora_mxfp4_linear_fwd(X.cuda(), W4, table, len(ranks), so, sa, r_max, 3, 8, S=S, keep_bits=keep)
    torch.cuda.synchronize()
    for s, a in enumerate(seg_ad):
        lo, hi = seg_off[s], seg_off[s + 1]
        if hi == lo:
            continue
        want, slack = layer_reference(X[lo:hi], W, As[a], Bs[a], dY[lo:hi], 0.5, ps[a], 3, 8 + lo * k)
        near(f"Y[{s}]", Y[lo:hi], want["Y"], slack["Y"])
        got = f64(S[lo:hi])
        assert (np.abs(got[:, :ranks[a]] - want["S"]) <= slack["S"] + 1e-30).all() and not got[:, ranks[a]:].any()
        assert torch.equal(keep[lo:hi], lf.lora_dropout_mask(3, 8 + lo * k, hi - lo, k, ps[a]))


@pytest.mark.gpu
@pytest.mark.parametrize("seg_off,seg_ad", [([0, -(1 << 33) + 5, 1 << 40, 20], [0, 1, 0]), ([0, 30, 10, 20], [1, 0, 1]),
                                            ([-7, 4, 4, 1 << 33], [0, 9, -3]), ([5, 6, 7, 8], [1, 1, 0])])
def test_bad_segment_tables_stay_in_bounds(seg_off, seg_ad):
    # offsets out of order, out of range, adapters that are not there: values of those rows are undefined, but
    # nothing outside the buffers' m rows is written
    m, k, n = 20, 264, 136
    g = torch.Generator().manual_seed(8)
    X, W4, W, _, _, dY = layer_case(m, k, n, 8, seed=8)
    As = [bf16_randn((k, r), 1.0, g).cuda() for r in (8, 40)]
    Bs = [bf16_randn((r, n), 1.0, g).cuda() for r in (8, 40)]
    table = lf.adapter_table(As, Bs, [1.0, 2.0], [0.1, 0.0])
    so = torch.tensor(seg_off, dtype=torch.int64, device="cuda")
    sa = torch.tensor(seg_ad, dtype=torch.int32, device="cuda")
    Y = torch.full((m + 80, n), 5.0, dtype=torch.bfloat16, device="cuda")
    S = torch.full((m + 80, 40), 5.0, device="cuda")
    keep = torch.full((m + 80, (k + 31) // 32), 5, dtype=torch.int32, device="cuda")
    mid = slice(40, 40 + m)
    lf.multi_lora_mxfp4_linear_fwd(X.cuda(), W4, table, 2, so, sa, 40, 3, 8, Y=Y[mid], S=S[mid], keep_bits=keep[mid])
    torch.cuda.synchronize()
    for t in (Y, S, keep):
        assert (t[:40] == 5).all() and (t[40 + m:] == 5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m", [5, 77, 300])
def test_mixed_short_segments(m):
    # many segments within one tile of rows, empty ones among them, ranks 1 to 256, unaligned matrices;
    # an infinity in one adapter's B and A shows in its own rows only
    k, n, ranks = 392, 136, [1, 256, 33, 7, 64]
    alphas, ps = [2.0, 0.25, 0.5, -1.0, 1.0], [0.0, 0.1, 0.2, 0.0, 0.05]
    g = torch.Generator().manual_seed(m + 1)
    X, W4, W, _, _, dY = layer_case(m, k, n, 8, seed=160 + m)
    As = [bf16_randn((k, r), k ** -0.5, g) for r in ranks]
    Bs = [bf16_randn((r, n), 0.02 ** 0.5, g) for r in ranks]
    cuts = torch.randint(0, m + 1, (24,), generator=g).sort().values.tolist()
    seg_off = [0, *cuts, m]
    seg_ad = torch.randint(0, 5, (len(seg_off) - 1,), generator=g).tolist()
    so = torch.tensor(seg_off, dtype=torch.int64, device="cuda")
    sa = torch.tensor(seg_ad, dtype=torch.int32, device="cuda")
    Ad, Bd = [offset_view(a) for a in As], [offset_view(b) for b in Bs]
    dAs, dBs = [torch.zeros_like(a) for a in Ad], [torch.zeros_like(b) for b in Bd]
    table = lf.adapter_table(Ad, Bd, alphas, ps, dAs, dBs)
    Xd, dYd = X.cuda(), dY.cuda()

    def run():
        Yb = torch.full((m + 2, n), 5.0, dtype=torch.bfloat16, device="cuda")
        dXb = torch.full((m + 2, k), 5.0, dtype=torch.bfloat16, device="cuda")
        _, S, keep = lf.multi_lora_mxfp4_linear_fwd(Xd, W4, table, 5, so, sa, 256, 3, 8, Y=Yb[:m])
        lf.multi_lora_mxfp4_linear_bwd(dYd, Xd, W4, table, 5, so, sa, S, keep, 256, dX=dXb[:m])
        torch.cuda.synchronize()
        assert (Yb[m:] == 5).all() and (dXb[m:] == 5).all()
        return Yb[:m], dXb[:m]

    Y, dX = run()
    for s, a in enumerate(seg_ad):
        lo, hi = seg_off[s], seg_off[s + 1]
        if hi > lo:
            want, slack = layer_reference(X[lo:hi], W, As[a], Bs[a], dY[lo:hi], alphas[a], ps[a], 3, 8 + lo * k)
            near(f"Y[{s}]", Y[lo:hi], want["Y"], slack["Y"])
            near(f"dX[{s}]", dX[lo:hi], want["dX"], slack["dX"])
    Y, dX = Y.clone(), dX.clone()
    hit = seg_ad[max(range(len(seg_ad)), key=lambda s: seg_off[s + 1] - seg_off[s])]
    Ad[hit][3, 0] = float("inf")
    Bd[hit][0, 5] = float("inf")
    Y2, dX2 = run()
    other = torch.ones(m, dtype=torch.bool)
    for s, a in enumerate(seg_ad):
        if a == hit:
            other[seg_off[s]:seg_off[s + 1]] = False
    assert torch.equal(Y2[other], Y[other]) and torch.equal(dX2[other], dX[other])
    assert not torch.isfinite(Y2[~other].float()).all()


# ---- use: streams, graphs, autograd ---------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("m,r,p", [(1, 16, 0.0), (1, 16, 0.1), (40, 64, 0.0), (700, 16, 0.1)])
def test_captured_layer_replays_match_eager(m, r, p):
    k, n, alpha = 520, 264, 2.0
    X, W4, W, A, B, dY = layer_case(m, k, n, r, seed=5)
    X, A, B, dY = X.cuda(), A.cuda(), B.cuda(), dY.cuda()

    def run():
        Y, S, keep = lf.lora_mxfp4_linear_fwd(X, W4, A, B, alpha, p, 9, 0)
        return (Y, S, lf.lora_mxfp4_frozen_fwd(X, W4), lf.lora_mxfp4_frozen_bwd(dY, W4),
                *lf.lora_mxfp4_linear_bwd(dY, X, W4, A, B, S, keep, alpha, p))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for rep in range(3):
        X.copy_(bf16_randn((m, k), 1.0, torch.Generator().manual_seed(100 + rep)))
        dY.copy_(bf16_randn((m, n), 1.0, torch.Generator().manual_seed(200 + rep)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for i, (a, b) in enumerate(zip(got, run())):
            assert torch.equal(a, b), f"replay {rep}: output {i}"


@pytest.mark.gpu
def test_two_streams_at_once():
    m, k, n, r = 40, 2056, 520, 16
    X, W4, W, A, B, _ = layer_case(m, k, n, r, seed=6)
    X2 = bf16_randn((m, k), 1.0, torch.Generator().manual_seed(8)).cuda()
    X, A, B = X.cuda(), A.cuda(), B.cuda()
    want = [lf.lora_mxfp4_linear_fwd(x, W4, A, B, 2.0, 0.0)[0] for x in (X, X2)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        got.append((lf.lora_mxfp4_linear_fwd(X, W4, A, B, 2.0, 0.0, stream=s1)[0],
                    lf.lora_mxfp4_linear_fwd(X2, W4, A, B, 2.0, 0.0, stream=s2)[0]))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 50, 600])
def test_captured_mixed_layers_side_by_side(m):
    # two graphs of the same shapes, replayed at once on two streams, with eager calls between
    k, n, ranks = 520, 264, [16, 40]
    g = torch.Generator().manual_seed(m)
    _, W4, _, _, _, _ = layer_case(m, k, n, 8, seed=12)
    so = torch.tensor([0, m // 2, m], dtype=torch.int64, device="cuda")
    sa = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    sides = []
    for i in range(2):
        As = [bf16_randn((k, r), k ** -0.5, g).cuda() for r in ranks]
        Bs = [bf16_randn((r, n), 0.02 ** 0.5, g).cuda() for r in ranks]
        dAs, dBs = [torch.zeros_like(a) for a in As], [torch.zeros_like(b) for b in Bs]
        table = lf.adapter_table(As, Bs, [2.0, 0.5], [0.1, 0.0], dAs, dBs)
        X, dY = bf16_randn((m, k), 1.0, g).cuda(), bf16_randn((m, n), 1.0, g).cuda()

        def run(X=X, dY=dY, table=table, dAs=dAs, dBs=dBs, As=As, Bs=Bs):
            Y, S, keep = lf.multi_lora_mxfp4_linear_fwd(X, W4, table, 2, so, sa, 40, 3, 8)
            dX = lf.multi_lora_mxfp4_linear_bwd(dY, X, W4, table, 2, so, sa, S, keep, 40)
            return Y, S, dX, *dAs, *dBs

        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        sides.append((run, stream, graph, out, X, dY))
    for rep in range(3):
        # (the segment table is read when the kernels run: a replay follows it)
        so[1] = (m // 2, 0, m)[rep]
        for _, _, _, _, X, dY in sides:
            X.copy_(bf16_randn(X.shape, 1.0, g))
            dY.copy_(bf16_randn(dY.shape, 1.0, g))
        torch.cuda.synchronize()
        for _, stream, graph, _, _, _ in sides:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for run, _, _, out, _, _ in sides:
            got = [t.clone() for t in out]
            for i, (a, b) in enumerate(zip(got, run())):
                assert torch.equal(a, b), f"replay {rep}: output {i}"
            torch.cuda.synchronize()


@pytest.mark.gpu
def test_no_rows():
    X, W4, W, A, B, dY = layer_case(4, 136, 72, 8, seed=1)
    X0, dY0, A, B = X[:0].cuda(), dY[:0].cuda(), A.cuda(), B.cuda()
    assert lf.lora_mxfp4_frozen_fwd(X0, W4).shape == (0, 72) and lf.lora_mxfp4_frozen_bwd(dY0, W4).shape == (0, 136)
    Y, S, keep = lf.lora_mxfp4_linear_fwd(X0, W4, A, B, 2.0, 0.0)
    dX, dA, dB = lf.lora_mxfp4_linear_bwd(dY0, X0, W4, A, B, S, keep, 2.0, 0.0)
    torch.cuda.synchronize()
    assert Y.shape == (0, 72) and dX.shape == (0, 136) and not dA.any() and not dB.any()


@pytest.mark.gpu
def test_weight_past_32_bits():
    # 2^32 values, codes past 2^31 bytes: the same 1024 columns over and over
    k, n, m, wide = 4096, 1 << 20, 3, 1024
    X, small, W, _, _, dY = layer_case(m, k, wide, 8, seed=91)
    rep = n // wide
    W4 = lf.Mxfp4Weight(small.codes.repeat(rep, 1, 1, 1), small.scales.repeat(rep, 1, 1), k, n)
    back = lf.lora_mxfp4_dequantize(W4)
    one = lf.lora_mxfp4_dequantize(small)
    assert torch.equal(back[:, -wide:], one) and torch.equal(back[-1].view(rep, wide), one[-1].expand(rep, wide))
    again = lf.lora_mxfp4_quantize(back)
    assert torch.equal(again.codes, W4.codes) and torch.equal(again.scales, W4.scales)
    del back, again
    Y = lf.lora_mxfp4_frozen_fwd(X.cuda(), W4).view(m, rep, wide)
    assert torch.equal(Y, Y[:, :1].expand(m, rep, wide))
    near("Y", Y[:, -1], f64(X) @ W, k * HALF * (np.abs(f64(X)) @ np.abs(W)))
    wider = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    wider[:, -wide:] = dY.cuda()
    dX = lf.lora_mxfp4_frozen_bwd(wider, W4)
    near("dX", dX, f64(dY) @ W.T, wide * HALF * (np.abs(f64(dY)) @ np.abs(W).T))  # (sums of zeros round nothing)


@pytest.mark.gpu
def test_no_rows_mixed():
    # no rows: the tables' gradients become zeros, and no scratch is needed for a weight that is not read
    k, n = 136, 72
    X, W4, W, _, _, dY = layer_case(4, k, n, 8, seed=1)
    As = [bf16_randn((k, r), 1.0, torch.Generator().manual_seed(r)).cuda() for r in (8, 40)]
    Bs = [bf16_randn((r, n), 1.0, torch.Generator().manual_seed(r)).cuda() for r in (8, 40)]
    dAs, dBs = [torch.full_like(a, 7.0) for a in As], [torch.full_like(b, 7.0) for b in Bs]
    table = lf.adapter_table(As, Bs, [1.0, 1.0], [0.0, 0.1], dAs, dBs)
    so = torch.zeros(3, dtype=torch.int64, device="cuda")
    sa = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    X0, dY0 = X[:0].cuda(), dY[:0].cuda()
    Y, S, keep = lf.multi_lora_mxfp4_linear_fwd(X0, W4, table, 2, so, sa, 40)
    dX = lf.multi_lora_mxfp4_linear_bwd(dY0, X0, W4, table, 2, so, sa, S, keep, 40)
    torch.cuda.synchronize()
    assert Y.shape == (0, n) and dX.shape == (0, k)
    assert not any(t.any() for t in (*dAs, *dBs))
    assert lf.lora_mxfp4_linear_bwd_workspace_size(0, 8192, 8192, 8) == _lib.lora_linear_bwd_workspace_size(0, 8192, 8192, 8)


@pytest.mark.gpu
def test_binding_rejects_on_the_gpu():
    X, W4, W, A, B, dY = layer_case(4, 136, 72, 8, seed=1)
    X, A, B = X.cuda(), A.cuda(), B.cuda()
    with pytest.raises(ValueError, match="do not hold"):
        lf.lora_mxfp4_frozen_fwd(X, W4._replace(n=200))
    with pytest.raises(ValueError, match="X must be"):
        lf.lora_mxfp4_frozen_fwd(X[:, :128].contiguous(), W4)
    with pytest.raises(ValueError, match="contiguous"):
        lf.lora_mxfp4_frozen_fwd(X[:, ::2].t().t(), W4)
    with pytest.raises(ValueError, match="B must be"):
        lf.lora_mxfp4_linear_fwd(X, W4, A, B[:4].contiguous(), 2.0, 0.0)
    with pytest.raises(ValueError, match="Y must be"):
        lf.lora_mxfp4_frozen_fwd(X, W4, Y=torch.empty(3, 72, dtype=torch.bfloat16, device="cuda"))
    need = lf.lora_mxfp4_linear_bwd_workspace_size(4, 136, 72, 8)
    _, S, keep = lf.lora_mxfp4_linear_fwd(X, W4, A, B, 2.0, 0.0)
    with pytest.raises(lf.LoraError, match="workspace"):
        lf.lora_mxfp4_linear_bwd(dY.cuda(), X, W4, A, B, S, keep, 2.0, 0.0,
                                 workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
def test_autograd_and_module_over_a_packed_weight():
    m, k, n, r = 150, 264, 136, 16
    X, W4, W, A, B, dY = layer_case(2 * m, k, n, r, seed=12)
    Wb = lf.lora_mxfp4_dequantize(W4)
    outs = []
    for weight in (W4, Wb):  # the same layer over the values in bf16 agrees within its own tolerance
        x = X.view(2, m, k).cuda().requires_grad_()
        a, b = A.cuda().requires_grad_(), B.cuda().requires_grad_()
        y = lf.lora_linear(x, weight, a, b, 2.0, 0.1, 11, 8)
        y.backward(dY.view(2, m, n).cuda())
        outs.append((y.detach(), x.grad, a.grad, b.grad))
    want, slack = layer_reference(X, W, A, B, dY, 2.0, 0.1, 11, 8)
    for o in outs:
        for name, t in zip(("Y", "dX", "dA", "dB"), o):
            near(name, t.reshape(want[name].shape), want[name], slack[name])

    layer = lf.LoraLinear(W4, r, 2.0, 0.0)
    with torch.no_grad():
        layer.B.copy_(B.cuda())
    twin = lf.LoraLinear(lf.lora_mxfp4_quantize(torch.zeros(k, n, dtype=torch.bfloat16, device="cuda")), r, 2.0)
    twin.load_state_dict(layer.state_dict())
    y = layer(X.cuda())
    assert torch.equal(y, twin(X.cuda()))
    y.float().square().sum().backward()
    assert layer.A.grad is not None and layer.B.grad is not None
    assert layer.weight_codes.dtype == torch.uint8


@pytest.mark.gpu
def test_mixed_autograd_over_a_packed_weight():
    m, k, n, ranks = 300, 264, 136, [16, 8]
    X, W4, W, _, _, dY = layer_case(m, k, n, 8, seed=14)
    g = torch.Generator().manual_seed(2)
    As = [bf16_randn((k, r), k ** -0.5, g).cuda().requires_grad_() for r in ranks]
    Bs = [bf16_randn((r, n), 0.02 ** 0.5, g).cuda().requires_grad_() for r in ranks]
    so = torch.tensor([0, 130, m], dtype=torch.int64, device="cuda")
    sa = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    x = X.cuda().requires_grad_()
    Y = lf.multi_lora_linear(x, W4, so, sa, As, Bs, [2.0, 1.0], [0.1, 0.0], 3, 16)
    Y.backward(dY.cuda())
    for lo, hi, a, alpha, p in ((0, 130, 1, 1.0, 0.0), (130, m, 0, 2.0, 0.1)):
        want, slack = layer_reference(X[lo:hi], W, As[a], Bs[a], dY[lo:hi], alpha, p, 3, 16 + lo * k)
        near("Y", Y[lo:hi], want["Y"], slack["Y"])
        near("dX", x.grad[lo:hi], want["dX"], slack["dX"])
        near("dA", As[a].grad, want["dA"], slack["dA"])
        near("dB", Bs[a].grad, want["dB"], slack["dB"])
