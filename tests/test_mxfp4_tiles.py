"""Every tile shape of the products over an MXFP4 weight, and the weight expanded for the
bf16 layer: with and without an adapter, in mixed batches, the contraction whole and split
over work-groups.  Rows, columns and the contraction end inside tiles, column groups and
blocks throughout.

The choice of a shape is a model of times; each case names the shapes that it is there for
(forward, then backward; None: expanded), and the timing pool says which ones ran, so that
a changed model cannot leave a shape untested unnoticed.

The references are torch products in 64 bits on the GPU over the unpacked weight (itself
tested against the format's definition in test_mxfp4.py); tolerances as derived there."""
import pytest
import torch

import lora_fine_tuning_amd as lf
from lora_fine_tuning_amd import _lib
from parity import bf16_randn, log, offset_view

BF, HALF, SPLIT = 2.0 ** -8, 2.0 ** -24, 2.0 ** -16
F64 = torch.float64

# m, k, n, then the tile and the slices of the contraction, forward and backward
FROZEN = [
    (5, 520, 136, "16x16", 1, "16x128", 1),
    (5, 8216, 136, "16x16", 9, "16x128", 1),
    (1, 520, 136, "4x16", 1, "16x128", 1),
    (2805, 136, 264, "48x128", 1, "32x128", 1),
    (258, 4760, 392, "48x128", 10, "48x128", 1),
    (4206, 264, 136, "48x128", 1, "64x128", 1),
    (481, 400, 1336, "32x128", 1, "64x128", 6),
    (1361, 1424, 216, "32x128", 1, "128x128", 1),
    (806, 464, 3192, "64x256", 1, "128x128", 9),
    (5508, 264, 136, "48x128", 1, "128x256", 1),
    (3, 5392, 1400, "4x16", 1, "128x256", 11),
    (5500, 136, 264, "64x256", 1, "48x128", 1),
    (676, 8936, 760, "64x256", 7, "128x256", 1),
    (6724, 136, 520, "128x256", 1, "64x128", 1),
    (2787, 4872, 728, "128x256", 3, None, 0),
    (8504, 136, 776, None, 0, "128x128", 1),
    (8308, 776, 136, "64x256", 1, None, 0),
    (2003, 4104, 4088, "128x256", 1, None, 0),
]

# m, k, n, r, ...
LAYER = [
    (1, 2920, 8136, 200, "4x16", 1, "16x128", 11),
    (1, 8208, 136, 5, "4x16", 9, "128x256", 3),
    (5, 8232, 136, 5, "16x16", 9, "16x128", 1),
    (853, 136, 328, 200, "48x128", 1, "16x128", 2),
    (698, 272, 376, 201, "48x128", 2, "32x128", 2),
    (5010, 136, 376, 200, "64x256", 1, "48x128", 1),
    (1003, 4184, 1144, 33, "64x128", 2, "128x256", 1),
    (997, 4176, 664, 200, "64x256", 5, "128x256", 1),
    (5484, 136, 552, 101, "128x256", 1, "48x128", 1),
    (3154, 3128, 296, 100, "128x256", 5, None, 0),
    (2003, 4104, 4088, 16, "128x256", 1, None, 0),
    (8630, 136, 792, 5, None, 0, "128x256", 3),
    (2363, 2664, 136, 200, "64x128", 6, None, 0),
    (3119, 392, 136, 16, "64x128", 2, "64x128", 1),
    (1323, 520, 280, 5, "64x128", 3, "64x128", 2),
    (4182, 400, 216, 100, "64x128", 1, "128x128", 1),
    (1131, 408, 1544, 8, "32x128", 1, "128x128", 7),
    (4099, 392, 136, 16, "64x128", 1, "128x256", 1),
    (1, 264, 136, 8, "4x32", 1, "128x256", 3),
]

# m, k, n, largest rank, segments, ...
MIXED = [
    (2, 5032, 7128, 200, 40, "4x16", 1, "16x128", 6),
    (1, 3160, 8728, 33, 3, "4x16", 1, "16x128", 9),
    (1, 8264, 136, 200, 40, "4x16", 9, "128x256", 3),
    (1, 8200, 136, 200, 3, "4x16", 9, "128x256", 3),
    (6, 8840, 136, 100, 40, "16x16", 9, "16x128", 1),
    (5, 8216, 136, 8, 40, "16x16", 9, "16x128", 1),
    (2894, 216, 280, 64, 40, "48x128", 1, "48x128", 2),
    (1436, 272, 296, 100, 40, "48x128", 2, "48x128", 2),
    (44, 520, 296, 200, 40, "48x128", 3, "128x256", 5),
    (1810, 488, 1144, 16, 40, "64x256", 1, "64x128", 2),
    (828, 3416, 1176, 64, 40, "64x256", 3, "128x256", 2),
    (1062, 1144, 4600, 100, 40, "128x256", 1, "128x256", 5),
    (4481, 1320, 392, 33, 40, "128x256", 3, "128x256", 1),
    (758, 136, 904, 100, 40, None, 0, "32x128", 4),
    (2904, 2152, 136, 16, 40, "48x128", 2, None, 0),
    (3080, 392, 136, 100, 3, "64x128", 2, "64x128", 1),
    (1133, 696, 264, 100, 8, "64x128", 3, "64x128", 2),
    (2365, 808, 248, 200, 8, "48x128", 2, "128x128", 1),
    (828, 1320, 1048, 33, 3, "64x128", 3, "128x128", 3),
    (4105, 392, 136, 33, 3, "64x128", 2, "128x256", 1),
    (1, 264, 136, 200, 8, "4x32", 1, "128x256", 3),
]

FORWARD = ["4x16", "4x32", "16x16", "16x64", "32x32", "32x128", "48x128", "64x128", "64x256", "128x256"]
BACKWARD = ["16x128", "32x128", "48x128", "64x128", "128x128", "128x256"]


class Ran:
    """Which products a block of calls launched, by the timing pool."""

    def __enter__(self):
        _lib.lora_profiling_enable(True, 256)
        return self

    def __exit__(self, *exc):
        def count(name):
            return _lib.lora_profiling_query(name)[0]

        self.forward = [t for t in FORWARD for _ in range(count("mxfp4_gemm " + t))]
        self.backward = [t for t in BACKWARD for _ in range(count("mxfp4_gemm_t " + t))]
        self.expanded = count("mxfp4_dequantize")
        _lib.lora_profiling_enable(False)

    def check(self, fwd, bwd):
        assert self.forward == [fwd] * (fwd is not None) and self.backward == [bwd] * (bwd is not None)
        assert self.expanded == (fwd is None) + (bwd is None)


def near(name, got, want, slack):
    """Every entry within half a bf16 step of `want` and `slack` of the sums before it."""
    got = got.to(F64)
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    over = (got - want).abs() - (BF * want.abs() + (1 + BF) * slack)
    worst = int(over.argmax())
    assert over.flatten()[worst] <= 0, (name, worst, float(got.flatten()[worst]), float(want.flatten()[worst]),
                                        float(slack.flatten()[worst]))


def inputs(m, k, n, seed):
    g = torch.Generator().manual_seed(seed)
    X, dY = bf16_randn((m, k), 1.0, g).cuda(), bf16_randn((m, n), 1.0, g).cuda()
    W4 = lf.lora_mxfp4_quantize(bf16_randn((k, n), k ** -0.5, g).cuda())
    return X, W4, lf.lora_mxfp4_dequantize(W4).to(F64), dY, g


def guarded(rows, cols, dtype=torch.bfloat16, fill=5.0):
    """(whole, middle): outputs whose neighbouring rows must stay as they were."""
    whole = torch.full((rows + 6, cols), fill, dtype=dtype, device="cuda")
    return whole, whole[3:3 + rows]


def untouched(*wholes):
    for w in wholes:
        fill = w[0, 0]
        assert fill in (5, 0x5A5A5A5A) and (w[:3] == fill).all() and (w[-3:] == fill).all()


def kept(seed, offset, m, k, p):
    """The dropout mask as 0 and 1, and the words that the forward stores."""
    words = lf.lora_dropout_mask(seed, offset, m, k, p)
    bits = words[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32) & 1
    return bits.reshape(m, -1)[:, :k].to(F64), words


def layer(X, W, A, B, dY, alpha, p, keep):
    """(outputs, slacks) of the layer's formulas."""
    (m, k), (r, n) = X.shape, B.shape
    x, a, b, dy = (t.to(F64) for t in (X, A, B, dY))
    scale = 1 / (1 - float(torch.tensor(p, dtype=torch.float32)))
    xd = x * keep * scale
    S, dS = xd @ a, alpha * (dy @ b.T)
    eS = (k + 2) * HALF * (xd.abs() @ a.abs())
    edS = (n + 2) * HALF * abs(alpha) * (dy.abs() @ b.abs().T)
    up, down = abs(alpha) * (S.abs() @ b.abs()), scale * (dS.abs() @ a.abs().T)
    da, db = xd.abs().T @ dS.abs(), S.abs().T @ dy.abs()
    out = {"S": S, "Y": x @ W + alpha * (S @ b), "dX": dy @ W.T + scale * keep * (dS @ a.T), "dA": xd.T @ dS,
           "dB": alpha * (S.T @ dy)}
    slack = {
        "S": eS,
        "Y": (k + r + 4) * HALF * (x.abs() @ W.abs() + up) + SPLIT * up + abs(alpha) * (eS @ b.abs()),
        "dX": (n + r + 4) * HALF * (dy.abs() @ W.abs().T + down) + SPLIT * down + scale * (edS @ a.abs().T),
        "dA": ((m + 4) * HALF + SPLIT) * da + xd.abs().T @ edS,
        "dB": abs(alpha) * (((m + 4) * HALF + SPLIT) * db + eS.T @ dy.abs()),
    }
    return out, slack


def test_the_cases_name_every_shape():
    for cases, at in ((FROZEN, 3), (LAYER, 4), (MIXED, 5)):
        fwd, bwd = {c[at:at + 2] for c in cases}, {c[at + 2:at + 4] for c in cases}
        for tile in ("4x16", "16x16", "48x128", "64x256", "128x256", None):
            assert any(t == tile for t, _ in fwd), tile
        for tile in ("16x128", "64x128", "128x128", "128x256", None):
            assert any(t == tile for t, _ in bwd), tile
        for tile in ("64x256", "128x256"):
            assert (tile, 1) in fwd and any(t == tile and s > 1 for t, s in fwd)
        assert ("128x256", 1) in bwd and any(t == "128x256" and s > 1 for t, s in bwd)


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n,fwd,fs,bwd,bs", FROZEN)
def test_frozen(m, k, n, fwd, fs, bwd, bs):
    log(f"frozen m={m} k={k} n={n}: {fwd} in {fs}, {bwd} in {bs}")
    X, W4, W, dY, _ = inputs(m, k, n, seed=m + n)
    Yw, Y = guarded(m, n)
    dXw, dX = guarded(m, k)
    with Ran() as ran:
        lf.lora_mxfp4_frozen_fwd(X, W4, Y=Y)
        lf.lora_mxfp4_frozen_bwd(dY, W4, dX=dX)
        torch.cuda.synchronize()
    ran.check(fwd, bwd)
    untouched(Yw, dXw)
    x, dy = X.to(F64), dY.to(F64)
    near("Y", Y, x @ W, k * HALF * (x.abs() @ W.abs()))
    near("dX", dX, dy @ W.T, n * HALF * (dy.abs() @ W.abs().T))


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(LAYER)))
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_layer(case, p):
    m, k, n, r, fwd, _, bwd, _ = LAYER[case]
    log(f"layer m={m} k={k} n={n} r={r} p={p}: {fwd}, {bwd}")
    X, W4, W, dY, g = inputs(m, k, n, seed=m + n + r)
    A, B = bf16_randn((k, r), k ** -0.5, g), bf16_randn((r, n), 0.02 ** 0.5, g)
    # every other adapter starts 2 bytes past a 16-byte boundary
    A, B = (offset_view(A), offset_view(B)) if case % 2 else (A.cuda(), B.cuda())
    alpha, seed, offset = -0.5, 7, 16
    Yw, Y = guarded(m, n)
    dXw, dX = guarded(m, k)
    Sw, S = guarded(m, r, torch.float32)
    Kw, K = guarded(m, (k + 31) // 32, torch.int32, 0x5A5A5A5A)
    with Ran() as ran:
        lf.lora_mxfp4_linear_fwd(X, W4, A, B, alpha, p, seed, offset, Y=Y, S=S, keep_bits=K)
        _, dA, dB = lf.lora_mxfp4_linear_bwd(dY, X, W4, A, B, S, K, alpha, p, dX=dX)
        torch.cuda.synchronize()
    ran.check(fwd, bwd)
    untouched(Yw, dXw, Sw, Kw)
    keep, words = kept(seed, offset, m, k, p)
    assert torch.equal(K, words)
    want, slack = layer(X, W, A, B, dY, alpha, p, keep)
    assert ((S.to(F64) - want["S"]).abs() <= slack["S"] + 1e-30).all()
    for name, t in (("Y", Y), ("dX", dX), ("dA", dA), ("dB", dB)):
        near(name, t, want[name], slack[name])
    # the same once more, without a mask to write where nothing is dropped, and without dX
    again = lf.lora_mxfp4_linear_fwd(X, W4, A, B, alpha, p, seed, offset)
    assert torch.equal(again[0], Y) and torch.equal(again[1], S)
    _, dA2, dB2 = lf.lora_mxfp4_linear_bwd(dY, X, W4, A, B, S, again[2], alpha, p, want_dX=False)
    assert torch.equal(dA2, dA) and torch.equal(dB2, dB)


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(MIXED)))
def test_mixed(case):
    m, k, n, r_max, nseg, fwd, _, bwd, _ = MIXED[case]
    log(f"mixed m={m} k={k} n={n} r_max={r_max} segments={nseg}: {fwd}, {bwd}")
    X, W4, W, dY, g = inputs(m, k, n, seed=m + n + nseg)
    ranks = [r_max, 1, max(1, r_max // 3)]
    alphas, ps = [2.0, -1.0, 0.5], [0.1, 0.0, 0.3]
    As = [bf16_randn((k, r), k ** -0.5, g).cuda() for r in ranks]
    Bs = [offset_view(bf16_randn((r, n), 0.02 ** 0.5, g)) for r in ranks]
    dAs, dBs = [torch.full_like(a, 7.0) for a in As], [torch.full_like(b, 7.0) for b in Bs]
    table = lf.adapter_table(As, Bs, alphas, ps, dAs, dBs)
    cuts = torch.randint(0, m + 1, (nseg - 1,), generator=g).sort().values.tolist()
    seg_off = [0, *cuts, m]
    seg_ad = torch.randint(0, 3, (nseg,), generator=g).tolist()
    so = torch.tensor(seg_off, dtype=torch.int64, device="cuda")
    sa = torch.tensor(seg_ad, dtype=torch.int32, device="cuda")
    Yw, Y = guarded(m, n)
    dXw, dX = guarded(m, k)
    Sw, S = guarded(m, r_max, torch.float32)
    Kw, K = guarded(m, (k + 31) // 32, torch.int32, 0x5A5A5A5A)
    with Ran() as ran:
        lf.multi_lora_mxfp4_linear_fwd(X, W4, table, 3, so, sa, r_max, 3, 8, Y=Y, S=S, keep_bits=K)
        lf.multi_lora_mxfp4_linear_bwd(dY, X, W4, table, 3, so, sa, S, K, r_max, dX=dX)
        torch.cuda.synchronize()
    ran.check(fwd, bwd)
    untouched(Yw, dXw, Sw, Kw)
    sums = [dict(dA=torch.zeros(a.shape, dtype=F64, device="cuda"), dB=torch.zeros(b.shape, dtype=F64, device="cuda"))
            for a, b in zip(As, Bs)]
    slacks = [{name: t.clone() for name, t in s.items()} for s in sums]
    for s, a in enumerate(seg_ad):
        lo, hi = seg_off[s], seg_off[s + 1]
        if hi == lo:
            continue
        keep, words = kept(3, 8 + lo * k, hi - lo, k, ps[a])
        assert torch.equal(K[lo:hi], words)
        want, slack = layer(X[lo:hi], W, As[a], Bs[a], dY[lo:hi], alphas[a], ps[a], keep)
        assert ((S[lo:hi, :ranks[a]].to(F64) - want["S"]).abs() <= slack["S"] + 1e-30).all()
        assert not S[lo:hi, ranks[a]:].any()
        near(f"Y[{s}]", Y[lo:hi], want["Y"], slack["Y"])
        near(f"dX[{s}]", dX[lo:hi], want["dX"], slack["dX"])
        for name in ("dA", "dB"):
            sums[a][name] += want[name]
            # (a segment's share counts the rows of all: each addition rounds a partial sum of the whole)
            slacks[a][name] += slack[name] * (m + 4) / (hi - lo + 4)
    for a in range(3):
        near(f"dA[{a}]", dAs[a], sums[a]["dA"], slacks[a]["dA"])
        near(f"dB[{a}]", dBs[a], sums[a]["dB"], slacks[a]["dB"])


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n,r", [(1 << 19, 72, 40, 8), ((1 << 19) + 5, 72, 40, 8), (3, 1 << 20, 24, 5), (3, (1 << 20) + 8, 24, 5),
                                     (3, 24, 1 << 20, 5), (3, 24, (1 << 21) + 8, 5)])
def test_sizes_around_the_packed_products_limits(m, k, n, r):
    # up to 2^19 rows, 2^20 of k and 2^21 columns (2^20 in the backward) the packed weight is read, past them it
    # is expanded
    log(f"limits m={m} k={k} n={n}")
    X, W4, W, dY, g = inputs(m, k, n, seed=5)
    A, B = bf16_randn((k, r), k ** -0.5, g).cuda(), bf16_randn((r, n), 0.02 ** 0.5, g).cuda()
    with Ran() as ran:
        Y, S, _ = lf.lora_mxfp4_linear_fwd(X, W4, A, B, 2.0, 0.0)
        dX, dA, dB = lf.lora_mxfp4_linear_bwd(dY, X, W4, A, B, S, None, 2.0, 0.0)
        torch.cuda.synchronize()
    past = m > 1 << 19 or k > 1 << 20 or n > 1 << 21
    assert not past or not (ran.forward or ran.backward) and ran.expanded == 2
    want, slack = layer(X, W, A, B, dY, 2.0, 0.0, torch.ones((), dtype=F64, device="cuda"))
    assert ((S.to(F64) - want["S"]).abs() <= slack["S"] + 1e-30).all()
    for name, t in (("Y", Y), ("dX", dX), ("dA", dA), ("dB", dB)):
        near(name, t, want[name], slack[name])
