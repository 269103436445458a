"""Every tile shape of the products over a weight of 4-bit integers, for groups of 32, 64
and 128 rows and of more, the contraction whole and split over work-groups, without an
adapter, with one and in mixed batches.  Rows, columns and the contraction end inside
tiles, column groups and blocks of 128 rows throughout.

The choice of a shape is a model of times; each case names the shape and the slices that
it is there for, and the timing pool says which ran, so that a changed model cannot leave
a shape untested unnoticed.  References and tolerances are test_int4.py's."""
import re

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as lf
from lora_fine_tuning_amd import _lib
from parity import bf16_randn, log
from test_int4 import case, f64, near, product, reference

# m, k, n, the tile, and whether the contraction is split
SHAPES = [
    (1, 520, 72, "int4_gemm 16x16", False), (3, 16392, 72, "int4_gemm 16x16", True), (1, 520, 8200, "int4_gemm 16x32", False),
    (3, 3000, 8200, "int4_gemm 16x32", False), (11, 136, 72, "int4_ring 16x32", False), (15, 8200, 1032, "int4_ring 16x32", True),
    (1, 136, 16392, "int4_ring 16x128", False), (20, 136, 72, "int4_ring 32x32", False), (27, 8200, 72, "int4_ring 32x32", True),
    (20, 264, 8200, "int4_ring 32x64", False), (29, 16392, 2056, "int4_ring 32x64", True), (33, 264, 72, "int4_ring 48x32", False),
    (47, 3000, 72, "int4_ring 48x32", True), (33, 264, 8200, "int4_ring 48x64", False), (45, 14344, 2056, "int4_ring 48x64", True),
    (50, 136, 72, "int4_ring 64x64", False), (55, 2056, 72, "int4_ring 64x64", True), (20, 136, 16392, "int4_ring 64x128", False),
    (55, 4104, 6152, "int4_ring 64x128", True), (65, 136, 72, "int4_ring 128x64", False), (141, 4104, 136, "int4_ring 128x64", True),
    (385, 520, 4104, "int4_ring 128x128", False), (141, 4104, 2056, "int4_ring 128x128", True),
    (1300, 520, 4104, "int4_ring 256x128", False), (550, 8, 9888, "int4_ring 256x128", False),
]
# the smallest groups that a case takes its tile for
LEAST = {(1, 520, 8200): 64, (3, 3000, 8200): 64, (55, 4104, 6152): 64, (1300, 520, 4104): 128, (550, 8, 9888): 128}


# the backward's: m, k, n, the tile, and whether the contraction (over n) is split
SHAPES_T = [
    (13, 136, 72, "int4_gemm_t 16x128", False), (13, 264, 4104, "int4_gemm_t 16x128", True), (600, 1032, 520, "int4_gemm_t 32x128", False),
    (20, 8200, 2056, "int4_gemm_t 32x128", True), (130, 8200, 2056, "int4_gemm_t 48x128", False), (40, 8200, 2056, "int4_gemm_t 48x128", True),
    (1500, 1032, 520, "int4_gemm_t 64x128", False), (60, 8200, 2056, "int4_gemm_t 64x128", True),
    (300, 8200, 2056, "int4_gemm_t 128x128", False), (2000, 264, 4104, "int4_gemm_t 128x128", True),
]


def ran(call, finish="int4_finish"):
    """The library's launches during `call`, by name, and whether a launch `finish` was among them."""
    lf.lora_profiling_enable(True, 64)
    lf.lora_profiling_reset()
    try:
        out = call()
        torch.cuda.synchronize()
        names = {s[3] for s in SHAPES + SHAPES_T}
        seen = {n for n in names if lf.lora_profiling_query(n)[0] > 0}
        split = lf.lora_profiling_query(finish)[0] > 0
    finally:
        lf.lora_profiling_enable(False)
    return out, seen, split


def test_every_shape_has_a_case():
    text = open(_lib.__file__.replace("_lib.py", "csrc/int4_gemm.hip")).read()
    names = set(re.findall(r'"(int4_(?:gemm|ring) \d+x\d+)"', text))
    assert names == {s[3] for s in SHAPES}
    text = open(_lib.__file__.replace("_lib.py", "csrc/int4_gemm_t.hip")).read()
    assert set(re.findall(r'"(int4_gemm_t \d+x\d+)"', text)) == {s[3] for s in SHAPES_T}


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n,tile,split,group", [(*s, g) for s in SHAPES for g in (32, 64, 128, 384) if g >= LEAST.get(s[:3], 32)])
def test_frozen(m, k, n, tile, split, group):
    log(f"frozen {m} x {k} x {n} group {group}: {tile}")
    X, W4, W, _, _, _ = case(m, k, n, 8, group, seed=m + k)
    Yb = torch.full((m + 2, n), 5.0, dtype=torch.bfloat16, device="cuda")
    _, seen, finish = ran(lambda: lf.lora_int4_frozen_fwd(X.cuda(), W4, Y=Yb[:m]))
    assert tile in seen and finish == split
    assert (Yb[m:] == 5).all()
    near("Y", Yb[:m], *product(m, f64(X), W))


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128, 384])
@pytest.mark.parametrize("m,k,n,tile,split", SHAPES_T)
def test_frozen_backward(m, k, n, tile, split, group):
    log(f"frozen backward {m} x {k} x {n} group {group}: {tile}")
    _, W4, W, _, _, dY = case(m, k, n, 8, group, seed=m + n)
    dXb = torch.full((m + 2, k), 5.0, dtype=torch.bfloat16, device="cuda")
    _, seen, finish = ran(lambda: lf.lora_int4_frozen_bwd(dY.cuda(), W4, dX=dXb[:m]), "mxfp4_join_down")
    assert tile in seen and finish == split
    assert (dXb[m:] == 5).all()
    dy = f64(dY)
    near("dX", dXb[:m], dy @ W[1].T, n * 2.0 ** -24 * (np.abs(dy) @ np.abs(W[1]).T))


@pytest.mark.gpu
@pytest.mark.parametrize("r,p", [(7, 0.0), (200, 0.1)])
@pytest.mark.parametrize("at", range(len(SHAPES_T)))
def test_layer_backward(at, r, p):
    m, k, n, _, _ = SHAPES_T[at]
    X, W4, W, A, B, dY = case(m, k, n, r, (32, 64, 128)[at % 3], seed=700 + at)
    Y, S, keep = lf.lora_int4_linear_fwd(X.cuda(), W4, A.cuda(), B.cuda(), 0.5, p, 5, 8)
    dX, dA, dB = lf.lora_int4_linear_bwd(dY.cuda(), X.cuda(), W4, A.cuda(), B.cuda(), S, keep, 0.5, p)
    want, slack = reference(X, W, A, B, dY, 0.5, p, 5, 8, m)
    for name, t in (("dX", dX), ("dA", dA), ("dB", dB)):
        near(name, t, want[name], slack[name])


@pytest.mark.gpu
@pytest.mark.parametrize("r,p", [(7, 0.0), (200, 0.1)])
@pytest.mark.parametrize("at", range(len(SHAPES)))
def test_layer(at, r, p):
    m, k, n, _, _ = SHAPES[at]
    group = max((32, 64, 128)[at % 3], LEAST.get((m, k, n), 32))
    X, W4, W, A, B, dY = case(m, k, n, r, group, seed=500 + at)
    Y, S, keep = lf.lora_int4_linear_fwd(X.cuda(), W4, A.cuda(), B.cuda(), 0.5, p, 5, 8)
    want, slack = reference(X, W, A, B, dY, 0.5, p, 5, 8, m)
    near("Y", Y, want["Y"], slack["Y"])
    assert (np.abs(f64(S) - want["S"]) <= slack["S"] + 1e-30).all()
    if p:
        assert torch.equal(keep, lf.lora_dropout_mask(5, 8, m, k, p))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 2, 9, 16, 17, 31, 48, 64, 100, 300])
@pytest.mark.parametrize("nseg", [1, 5, 70, 400])
def test_segments(m, nseg):
    # more segments than rows (most are empty), more than the product's launch forms S for, an adapter with rank 256
    k, n, ranks = 1032, 136, [256, 8, 33, 1, 64]
    alphas, ps = [0.25, 2.0, 0.5, -1.0, 1.0], [0.1, 0.0, 0.2, 0.0, 0.05]
    g = torch.Generator().manual_seed(m + nseg)
    X, W4, W, _, _, dY = case(m, k, n, 8, 64, seed=m)
    As = [bf16_randn((k, r), k ** -0.5, g) for r in ranks]
    Bs = [bf16_randn((r, n), 0.02 ** 0.5, g) for r in ranks]
    Ad, Bd = [a.cuda() for a in As], [b.cuda() for b in Bs]
    table = lf.adapter_table(Ad, Bd, alphas, ps)
    cuts = torch.randint(0, m + 1, (nseg - 1,), generator=g).sort().values.tolist()
    seg_off, seg_ad = [0, *cuts, m], torch.randint(0, 5, (nseg,), generator=g).tolist()
    so = torch.tensor(seg_off, dtype=torch.int64, device="cuda")
    sa = torch.tensor(seg_ad, dtype=torch.int32, device="cuda")
    S = torch.full((m, 256), float("nan"), device="cuda")
    Y, S, keep = lf.multi_lora_int4_linear_fwd(X.cuda(), W4, table, 5, so, sa, 256, 3, 8, S=S)
    again = lf.multi_lora_int4_linear_fwd(X.cuda(), W4, table, 5, so, sa, 256, 3, 8)
    torch.cuda.synchronize()
    assert torch.equal(Y, again[0]) and torch.equal(S, again[1]) and torch.equal(keep, again[2])
    for s, a in enumerate(seg_ad):
        lo, hi = seg_off[s], seg_off[s + 1]
        if hi > lo:
            want, slack = reference(X[lo:hi], W, As[a], Bs[a], dY[lo:hi], alphas[a], ps[a], 3, 8 + lo * k, m)
            near(f"Y[{s}]", Y[lo:hi], want["Y"], slack["Y"])
            got = f64(S[lo:hi])
            assert (np.abs(got[:, :ranks[a]] - want["S"]) <= slack["S"] + 1e-30).all() and not got[:, ranks[a]:].any()
            assert torch.equal(keep[lo:hi], lf.lora_dropout_mask(3, 8 + lo * k, hi - lo, k, ps[a]))


@pytest.mark.gpu
def test_infinite_adapters_stay_in_their_rows():
    m, k, n = 24, 264, 136
    g = torch.Generator().manual_seed(3)
    X, W4, _, _, _, _ = case(m, k, n, 8, 32, seed=4)
    As = [bf16_randn((k, r), k ** -0.5, g).cuda() for r in (8, 40)]
    Bs = [bf16_randn((r, n), 1.0, g).cuda() for r in (8, 40)]
    table = lf.adapter_table(As, Bs, [1.0, 2.0], [0.0, 0.0])
    so = torch.tensor([0, 5, 6, 20, m], dtype=torch.int64, device="cuda")
    sa = torch.tensor([0, 1, 0, 1], dtype=torch.int32, device="cuda")
    Y = lf.multi_lora_int4_linear_fwd(X.cuda(), W4, table, 2, so, sa, 40)[0].clone()
    As[1][3, 0] = float("inf")
    Bs[1][5, 7] = float("nan")
    Y2 = lf.multi_lora_int4_linear_fwd(X.cuda(), W4, table, 2, so, sa, 40)[0]
    other = torch.ones(m, dtype=torch.bool, device="cuda")
    other[5:6] = other[20:] = False
    assert torch.equal(Y2[other], Y[other]) and not torch.isfinite(Y2[~other].float()).all(1).any()
