"""The layers over a weight of 4-bit integers in every tile shape of their products: with one
adapter, which the wide tiles (128 and 256 rows) add in their own epilogue where the contraction
is not split and a finishing launch adds otherwise, and in mixed batches; the backward likewise.

Each case names its shape, and the timing pool says which ran and that the weight was not
expanded, so the one reference that holds is the packed weight's.  References and tolerances are
test_int4.py's."""
import re

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as lf
from lora_fine_tuning_amd import _lib
from parity import bf16_randn, log
from test_int4 import case, f64, near, reference

# one adapter, more than 64 rows: m, k, n, group, r, the tile, and whether the contraction is split.  Ranks
# take one and several steps of 32, whole and odd ones (S is read 16 bytes at a time, or 4)
WIDE = [
    (100, 136, 136, 32, 7, "128x64", False), (300, 264, 136, 128, 16, "128x64", False), (65, 136, 6152, 128, 40, "128x64", False),
    (65, 520, 8200, 32, 37, "128x64", False), (129, 264, 6152, 64, 63, "128x64", False),
    (65, 136, 72, 32, 200, "128x64", True), (65, 520, 72, 128, 7, "128x64", True), (129, 1032, 136, 64, 33, "128x64", True),
    (129, 136, 8200, 128, 7, "128x128", False), (65, 136, 16392, 64, 7, "128x128", False), (300, 1032, 8200, 128, 16, "128x128", False),
    (300, 1032, 8200, 128, 64, "128x128", False), (129, 264, 12296, 384, 40, "128x128", False), (129, 520, 8200, 64, 37, "128x128", False),
    (65, 1032, 16392, 32, 40, "128x128", False),
    (65, 264, 6152, 128, 200, "128x128", True), (65, 1032, 6152, 64, 16, "128x128", True), (65, 264, 6152, 32, 40, "128x128", True),
    (129, 520, 24584, 128, 7, "256x128", False), (129, 1032, 24584, 128, 40, "256x128", False),
    (129, 1032, 6152, 128, 200, "256x128", True), (129, 1032, 6152, 384, 203, "256x128", True),
]

# up to 64 rows, where S is formed beside the product: m, k, n, group, the tile (each whole, then split)
FEW = [
    (1, 520, 72, 64, "int4_gemm 16x16"), (1, 1032, 72, 128, "int4_gemm 16x16"), (1, 520, 8200, 64, "int4_gemm 16x32"),
    (1, 2056, 2056, 128, "int4_gemm 16x32"), (1, 136, 16392, 128, "int4_ring 16x128"), (1, 2056, 16392, 64, "int4_ring 16x128"),
    (11, 136, 72, 32, "int4_ring 16x32"), (11, 520, 72, 64, "int4_ring 16x32"), (20, 136, 72, 64, "int4_ring 32x32"),
    (20, 520, 72, 128, "int4_ring 32x32"), (20, 264, 8200, 128, "int4_ring 32x64"), (20, 1032, 4104, 64, "int4_ring 32x64"),
    (33, 264, 72, 128, "int4_ring 48x32"), (33, 520, 72, 32, "int4_ring 48x32"), (33, 264, 8200, 64, "int4_ring 48x64"),
    (33, 520, 4104, 128, "int4_ring 48x64"), (50, 136, 72, 32, "int4_ring 64x64"), (50, 264, 72, 128, "int4_ring 64x64"),
    (20, 136, 16392, 128, "int4_ring 64x128"), (33, 520, 8200, 64, "int4_ring 64x128"),
]

# mixed batches of more than 64 rows: m, k, n, group, the largest rank, segments, the tile (whole and split)
MIXED = [
    (65, 8, 72, 128, 64, 4, "128x64"), (65, 136, 72, 32, 64, 4, "128x64"), (300, 1032, 136, 64, 200, 5, "128x64"),
    (129, 8, 8200, 64, 64, 4, "128x128"), (129, 520, 4104, 32, 64, 4, "128x128"), (300, 1032, 8200, 128, 64, 4, "128x128"),
    (129, 1032, 4104, 64, 256, 3, "128x128"), (129, 8, 16392, 128, 64, 4, "256x128"), (129, 1032, 8200, 128, 64, 4, "256x128"),
    (129, 1032, 8200, 384, 64, 4, "256x128"),
]

# the backward: m, k, n, group, the tile (each split, then whole)
BACK = [
    (13, 264, 4104, 64, "16x128"), (13, 136, 72, 32, "16x128"), (20, 8200, 2056, 128, "32x128"), (2600, 136, 72, 32, "32x128"),
    (40, 8200, 2056, 64, "48x128"), (100, 8200, 136, 128, "48x128"), (300, 1032, 2056, 128, "64x128"), (2600, 520, 136, 64, "64x128"),
    (900, 1032, 520, 128, "128x128"), (100, 8200, 72, 128, "128x128"),
]


def tiles():
    """Every tile's name in the sources."""
    text = "".join(open(_lib.__file__.replace("_lib.py", f"csrc/{f}.hip")).read() for f in ("int4_gemm", "int4_gemm_t"))
    return set(re.findall(r'"(int4_(?:gemm|ring|gemm_t) \d+x\d+)"', text))


def launches(call):
    """The call's result, and how often each of the library's launches ran in it."""
    names = [*tiles(), "int4_finish", "int4_dequantize", "int4_s", "mxfp4_join_up", "mxfp4_join_down"]
    lf.lora_profiling_enable(True, 64)
    lf.lora_profiling_reset()
    try:
        out = call()
        torch.cuda.synchronize()
        return out, {n: lf.lora_profiling_query(n)[0] for n in names if lf.lora_profiling_query(n)[0] > 0}
    finally:
        lf.lora_profiling_enable(False)


def test_every_shape_has_a_case():
    forward = {f"int4_ring {t[5]}" for t in WIDE}
    assert forward | {t[-1] for t in FEW} | {f"int4_gemm_t {t[-1]}" for t in BACK} == tiles()
    assert {f"int4_ring {t[-1]}" for t in MIXED} == forward
    assert {(t[5], t[6]) for t in WIDE} == {(t, s) for t in ("128x64", "128x128", "256x128") for s in (False, True)}


@pytest.mark.gpu
@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("m,k,n,group,r,tile,split", WIDE)
def test_one_adapter(m, k, n, group, r, tile, split, p):
    log(f"layer {m} x {k} x {n} r {r} group {group}: {tile}")
    X, W4, W, A, B, dY = case(m, k, n, r, group, seed=m + n + r)
    Yb = torch.full((m + 2, n), 5.0, dtype=torch.bfloat16, device="cuda")
    (_, S, keep), seen = launches(lambda: lf.lora_int4_linear_fwd(X.cuda(), W4, A.cuda(), B.cuda(), 0.5, p, 5, 8, Y=Yb[:m]))
    assert seen == {f"int4_ring {tile}": 1, **({"int4_finish": 1} if split else {})}
    assert (Yb[m:] == 5).all()
    want, slack = reference(X, W, A, B, dY, 0.5, p, 5, 8, 1)
    near("Y", Yb[:m], want["Y"], slack["Y"])
    assert (np.abs(f64(S) - want["S"]) <= slack["S"] + 1e-30).all()
    if p:
        assert torch.equal(keep, lf.lora_dropout_mask(5, 8, m, k, p))


@pytest.mark.gpu
@pytest.mark.parametrize("r,p", [(7, 0.1), (40, 0.0)])
@pytest.mark.parametrize("m,k,n,group,tile", FEW)
def test_few_rows_one_adapter(m, k, n, group, tile, r, p):
    log(f"layer {m} x {k} x {n} r {r} group {group}: {tile}")
    X, W4, W, A, B, dY = case(m, k, n, r, group, seed=m + n + r)
    (Y, S, keep), seen = launches(lambda: lf.lora_int4_linear_fwd(X.cuda(), W4, A.cuda(), B.cuda(), 0.5, p, 5, 8))
    assert seen == {tile: 1, "int4_finish": 1}
    want, slack = reference(X, W, A, B, dY, 0.5, p, 5, 8, 1)
    near("Y", Y, want["Y"], slack["Y"])
    assert (np.abs(f64(S) - want["S"]) <= slack["S"] + 1e-30).all()
    if p:
        assert torch.equal(keep, lf.lora_dropout_mask(5, 8, m, k, p))


def mixed(m, k, n, group, r_max, nseg, seed):
    """A batch of segments (some empty) over three adapters, the last of rank r_max."""
    g = torch.Generator().manual_seed(seed)
    ranks, alphas, ps = [min(8, r_max), max(1, r_max // 2 - 3), r_max], [0.5, 2.0, -1.0], [0.1, 0.0, 0.2]
    As = [bf16_randn((k, r), k ** -0.5, g) for r in ranks]
    Bs = [bf16_randn((r, n), 0.02 ** 0.5, g) for r in ranks]
    cuts = torch.randint(0, m + 1, (nseg - 1,), generator=g).sort().values.tolist()
    return As, Bs, alphas, ps, [0, *cuts, m], [(i + 2) % 3 for i in range(nseg)]


def check_mixed(m, k, n, group, r_max, nseg, expect):
    X, W4, W, _, _, dY = case(m, k, n, 8, group, seed=m + n)
    As, Bs, alphas, ps, seg_off, seg_ad = mixed(m, k, n, group, r_max, nseg, m + nseg)
    Ad, Bd = [a.cuda() for a in As], [b.cuda() for b in Bs]
    table = lf.adapter_table(Ad, Bd, alphas, ps)
    so = torch.tensor(seg_off, dtype=torch.int64, device="cuda")
    sa = torch.tensor(seg_ad, dtype=torch.int32, device="cuda")
    S = torch.full((m, r_max), float("nan"), device="cuda")
    (Y, S, keep), seen = launches(lambda: lf.multi_lora_int4_linear_fwd(X.cuda(), W4, table, 3, so, sa, r_max, 3, 8, S=S))
    assert seen == expect
    for s, a in enumerate(seg_ad):
        lo, hi = seg_off[s], seg_off[s + 1]
        if hi > lo:
            want, slack = reference(X[lo:hi], W, As[a], Bs[a], dY[lo:hi], alphas[a], ps[a], 3, 8 + lo * k, 1)
            near(f"Y[{s}]", Y[lo:hi], want["Y"], slack["Y"])
            got, r = f64(S[lo:hi]), As[a].shape[1]
            assert (np.abs(got[:, :r] - want["S"]) <= slack["S"] + 1e-30).all() and not got[:, r:].any()
            assert torch.equal(keep[lo:hi], lf.lora_dropout_mask(3, 8 + lo * k, hi - lo, k, ps[a]))


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n,group,r_max,nseg,tile", MIXED)
def test_mixed(m, k, n, group, r_max, nseg, tile):
    log(f"mixed {m} x {k} x {n} r {r_max} group {group}: {tile}")
    check_mixed(m, k, n, group, r_max, nseg, {"int4_s": 1, f"int4_ring {tile}": 1, "mxfp4_join_up": 1})


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n,group,tile", FEW)
def test_few_rows_mixed(m, k, n, group, tile):
    log(f"mixed {m} x {k} x {n} group {group}: {tile}")
    check_mixed(m, k, n, group, 64, 4, {tile: 1, "int4_finish": 1})


@pytest.mark.gpu
@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("r,p", [(7, 0.1), (40, 0.0), (200, 0.1)])
@pytest.mark.parametrize("m,k,n,group,tile", BACK)
def test_backward(m, k, n, group, tile, r, p, saved):
    log(f"backward {m} x {k} x {n} r {r} group {group} saved {saved}: {tile}")
    X, W4, W, A, B, dY = case(m, k, n, r, group, seed=m + n + r)
    Ad, Bd, Xd, dYd = A.cuda(), B.cuda(), X.cuda(), dY.cuda()
    _, S, keep = lf.lora_int4_linear_fwd(Xd, W4, Ad, Bd, 0.5, p, 5, 8)
    X8 = lf.lora_mxint8_quantize(Xd)
    dXb = torch.full((m + 2, k), 5.0, dtype=torch.bfloat16, device="cuda")

    def call():
        if saved:
            return lf.lora_mxint8_linear_bwd(dYd, X8, W4, Ad, Bd, S, keep, 0.5, p, dX=dXb[:m])
        return lf.lora_int4_linear_bwd(dYd, Xd, W4, Ad, Bd, S, keep, 0.5, p, dX=dXb[:m])

    (_, dA, dB), seen = launches(call)
    assert seen == {f"int4_gemm_t {tile}": 1, "mxfp4_join_down": 1}
    assert (dXb[m:] == 5).all()
    want, slack = reference(X, W, A, B, dY, 0.5, p, 5, 8, 1)
    near("dX", dXb[:m], want["dX"], slack["dX"])
    near("dB", dB, want["dB"], slack["dB"])
    if saved:
        want, slack = reference(lf.lora_mxint8_dequantize(X8).cpu(), W, A, B, dY, 0.5, p, 5, 8, 1)
    near("dA", dA, want["dA"], slack["dA"])
