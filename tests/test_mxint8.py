"""A layer's input saved in 8 bits (MXINT8), and the layer's backward from it.

The format's reference is written here from its definition, in 64 bits with numpy.

Tolerances, derived: saving and reading back are exact (every value that codes and
scales stand for is a bf16), so the backward from a saved input is the bf16 layer's
over that input: where the same kernels run (ranks that are multiples of 8; dX without a
mask, or of a multiple of 128 columns), bit for bit, and otherwise within test_mxfp4.layer_reference's slack of the 64-bit
formulas.  dX and dB do not read the input: their formulas are those over X itself,
which S is of.
"""
import gc
import os

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as lf
from lora_fine_tuning_amd import _lib
from parity import bf16_randn, log, offset_view
from test_mxfp4 import f64, layer_reference, near

FAKE = 0x10000  # aligned, never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
BF16, MXFP4, INT4 = 0, 1, 2


# ---- the format, from its definition ---------------------------------------------------------

def ref_save(X):
    """(codes (m, KB, 32), scale bytes (m, KB)) of a float64 matrix of bf16 values."""
    m, k = X.shape
    kb = -(-k // 128) * 4
    x = np.zeros((m, kb * 32))
    x[:, :k] = X
    x = x.reshape(m, kb, 32)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(np.isfinite(x), x, 0.0)
    top = np.abs(x).max(-1)
    some = top > 0
    e = np.zeros((m, kb))
    e[some] = np.clip(np.frexp(top[some])[1] - 1 - 6, -120, 121)
    c = np.clip(np.rint(x / 2.0 ** e[..., None]), -127, 127)
    c[bad] = 0
    return c.astype(np.int8), np.where(bad, 255, e + 127).astype(np.uint8)


def ref_values(codes, scales, k):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(float) - 127))
    return (codes * s[..., None]).reshape(codes.shape[0], -1)[:, :k]


def check_save(X):
    c, s = ref_save(f64(X))
    X8 = lf.lora_mxint8_quantize(X.cuda())
    torch.cuda.synchronize()
    assert np.array_equal(X8.codes.cpu().numpy(), c) and np.array_equal(X8.scales.cpu().numpy(), s)
    back = f64(lf.lora_mxint8_dequantize(X8))
    want = ref_values(c, s, X.shape[1])
    assert np.array_equal(back, want, equal_nan=True)
    return X8, back


def test_reference_error_bound():
    # every value a bf16 and off by half a step of its block at most: 1/128 of the largest (a / 2^e is at least 64)
    rng = np.random.default_rng(0)
    X = f64(torch.from_numpy(rng.standard_normal((50, 392)) * 2.0 ** rng.integers(-30, 30, (50, 1))).bfloat16())
    c, s = ref_save(X)
    V = ref_values(c, s, 392)
    assert np.array_equal(f64(torch.from_numpy(V).bfloat16()), V)
    step = np.repeat(2.0 ** (s.astype(float) - 127), 32, 1)[:, :392]
    assert (np.abs(V - X) <= step / 2).all()
    top = np.abs(np.pad(X, ((0, 0), (0, 120))).reshape(50, 16, 32)).max(-1)
    assert (np.abs(V - X) <= np.repeat(top, 32, 1)[:, :392] / 128).all()
    c2, s2 = ref_save(V)
    assert np.array_equal(ref_values(c2, s2, 392), V)


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
    for m, k, want in ((0, 8, 0), (1, 8, 128), (3, 128, 3 * 128), (3, 136, 3 * 256), (8192, 28672, 8192 * 28672)):
        assert lib.lora_mxint8_codes_size(m, k) == want and lib.lora_mxint8_scales_size(m, k) == want // 32
    assert lib.lora_mxint8_codes_size(-1, 8) == 0 and lib.lora_mxint8_codes_size(8, 0) == 0
    for kind, layer in ((BF16, _lib.lora_linear_bwd_workspace_size), (MXFP4, lf.lora_mxfp4_linear_bwd_workspace_size),
                        (INT4, lambda m, k, n, r: lf.lora_int4_linear_bwd_workspace_size(m, k, n, 64, r))):
        for r in (8, 13, 200):
            assert lf.lora_mxint8_linear_bwd_workspace_size(kind, 64, 100, 264, 136, r) >= layer(100, 264, 136, r)
    assert lf.lora_mxint8_linear_bwd_workspace_size(BF16, 0, 100, 264, 136, 0) == 0
    assert lf.multi_lora_mxint8_bwd_workspace_size(BF16, 0, 100, 264, 136, 300, 2, 2) == 0


def test_save_rejects(lib):
    for f in (lib.lora_mxint8_quantize, lambda X, m, k, c, s, st: lib.lora_mxint8_dequantize(c, s, m, k, X, st)):
        ok = dict(X=FAKE, m=4, k=64, c=FAKE, s=FAKE)
        for kw in (dict(X=None), dict(X=FAKE + 8), dict(k=60), dict(k=0), dict(m=-1), dict(c=None), dict(c=FAKE + 8), dict(s=FAKE + 2),
                   dict(s=None), dict(m=1 << 30, k=1 << 20)):
            a = {**ok, **kw}
            assert f(a["X"], a["m"], a["k"], a["c"], a["s"], None) == INVALID, kw
        assert f(None, 0, 64, None, None, None) == 0


@pytest.mark.parametrize("kind", [BF16, MXFP4, INT4])
def test_backward_rejects(lib, kind):
    F, big = FAKE, 1 << 40

    def bwd(**kw):
        a = dict(dY=F, c=F, s=F, kind=kind, W=F, Ws=F, group=64, A=F, B=F, S=F, keep=F, m=64, k=64, n=64, r=8, p=0.1, dX=F, dA=F, dB=F,
                 ws=F, wsb=big)
        a.update(kw)
        return lib.lora_mxint8_linear_bwd(a["dY"], a["c"], a["s"], a["kind"], a["W"], a["Ws"], a["group"], a["A"], a["B"], a["S"],
                                          a["keep"], a["m"], a["k"], a["n"], a["r"], 1.0, a["p"], a["dX"], a["dA"], a["dB"], a["ws"],
                                          a["wsb"], None)

    for kw in (dict(dY=None), dict(c=None), dict(c=F + 8), dict(s=F + 2), dict(kind=3), dict(kind=-1), dict(W=None), dict(W=F + 8),
               dict(A=None), dict(B=None), dict(dA=None), dict(dB=None), dict(S=None), dict(S=F + 2), dict(keep=None), dict(keep=F + 2),
               dict(r=0), dict(r=257), dict(p=1.0), dict(p=float("nan")), dict(dX=F + 2), dict(k=20), dict(n=12), dict(m=-1),
               dict(ws=None)):
        assert bwd(**kw) == INVALID, kw
    if kind != BF16:
        assert bwd(Ws=None) == INVALID and bwd(Ws=F + 8) == INVALID
    if kind == INT4:
        assert bwd(group=96) == INVALID and bwd(group=0) == INVALID
    for r in (8, 13, 200):
        need = lib.lora_mxint8_linear_bwd_workspace_size(kind, 64, 64, 64, 64, r)
        assert bwd(r=r, wsb=need - 1) == WORKSPACE and bwd(r=r, wsb=need - 1, dX=None) == WORKSPACE
    assert bwd(r=256, k=1 << 22) == UNSUPPORTED and bwd(r=256, n=1 << 22) == UNSUPPORTED

    def multi(**kw):
        a = dict(dY=F, c=F, s=F, kind=kind, W=F, Ws=F, group=64, tab=F, na=2, so=F, sa=F, ns=1, S=F, keep=F, m=64, k=64, n=64, r=16, dX=F,
                 ws=F, wsb=big)
        a.update(kw)
        return lib.multi_lora_mxint8_linear_bwd(a["dY"], a["c"], a["s"], a["kind"], a["W"], a["Ws"], a["group"], a["tab"], a["na"],
                                                a["so"], a["sa"], a["ns"], a["S"], a["keep"], a["m"], a["k"], a["n"], a["r"], a["dX"],
                                                a["ws"], a["wsb"], None)

    for kw in (dict(dY=None), dict(c=None), dict(s=F + 2), dict(kind=7), dict(W=F + 8), dict(tab=None), dict(na=0), dict(so=None),
               dict(sa=None), dict(ns=0), dict(S=None), dict(keep=None), dict(r=300), dict(r=0), dict(dX=F + 8), dict(k=20), dict(ws=None)):
        assert multi(**kw) == INVALID, kw
    assert multi(wsb=0) == WORKSPACE and multi(r=256, n=1 << 22) == UNSUPPORTED


def test_binding_rejects():
    X = torch.zeros(3, 64, dtype=torch.bfloat16)
    X8 = lf.Mxint8Input(torch.zeros(3, 4, 32, dtype=torch.int8), torch.zeros(3, 4, dtype=torch.uint8), 64)
    with pytest.raises(TypeError, match="bfloat16"):
        lf.lora_mxint8_quantize(X.float())
    with pytest.raises(TypeError, match="Mxint8Input"):
        lf.lora_mxint8_dequantize(X)
    with pytest.raises(ValueError, match="do not hold"):
        lf.lora_mxint8_dequantize(X8._replace(k=136))
    with pytest.raises(ValueError, match="do not hold"):
        lf.lora_mxint8_dequantize(X8._replace(scales=X8.scales[:2]))
    with pytest.raises(TypeError, match="int8"):
        lf.lora_mxint8_dequantize(X8._replace(codes=X8.codes.int()))
    with pytest.raises(ValueError, match="device"):
        lf.lora_mxint8_dequantize(X8)
    W, A, B = (torch.zeros(s, dtype=torch.bfloat16) for s in ((64, 64), (64, 8), (8, 64)))
    with pytest.raises(ValueError, match="X8 holds"):
        lf.lora_linear(X[:2], W, A, B, 1.0, X8=X8)
    with pytest.raises(TypeError, match="Mxint8Input"):
        lf.lora_linear(X, W, A, B, 1.0, X8=X)
    with pytest.raises(ValueError, match="save_bits"):
        lf.LoraLinear(W, 8, 1.0, save_bits=4)


# ---- saving (GPU) ---------------------------------------------------------------------------------

SAVE = [(1, 8), (1, 128), (3, 136), (7, 2048), (33, 2056), (5, 4104), (333, 1032), (64, 14336), (2, 28672), (1000, 24)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,k", SAVE)
def test_save_matches_definition(m, k):
    log(f"save {m}x{k}")
    g = torch.Generator().manual_seed(m + k)
    X = bf16_randn((m, k), 1.0, g)
    X[:, ::17] *= 30.0
    check_save(X)


@pytest.mark.gpu
def test_save_every_bf16():
    # each finite bf16 among 31 zeros, and beside larger ones, in both signs
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    vals = bits[torch.isfinite(bits)]
    X = torch.zeros(vals.numel(), 32, dtype=torch.bfloat16)
    X[:, 3] = vals
    check_save(X)
    for shift in (0.5, 1.0, 3.0, 129.0):
        X[:, 9] = (vals.double() * shift).clamp(-3.3e38, 3.3e38).bfloat16()
        check_save(X)


@pytest.mark.gpu
def test_save_special_values():
    X = bf16_randn((9, 168), 1.0, torch.Generator().manual_seed(1))
    X[0] = 0.0
    X[1] = -0.0
    X[2] = 2.0 ** -133
    X[3] = 3.3895313892515355e38
    X[4, :32] = torch.linspace(-127.5, 127.5, 32).bfloat16()
    X[4, 32:64] = 127.5
    X[5, 3], X[6, 40], X[7, 167] = float("inf"), float("nan"), -float("inf")
    X[8, :64] = 2.0 ** -122
    X8, back = check_save(X)
    bad = np.isnan(back)
    assert bad[5, :32].all() and bad[6, 32:64].all() and bad[7, 160:].all() and bad.sum() == 32 + 32 + 8


@pytest.mark.gpu
def test_every_scale_byte_reads_as_its_power():
    codes = torch.arange(-127, 129).clamp(-127, 127).to(torch.int8).view(8, 1, 32).expand(8, 256, 32).contiguous()
    scales = torch.arange(256).to(torch.uint8).expand(8, 256).contiguous()
    back = lf.lora_mxint8_dequantize(lf.Mxint8Input(codes.cuda(), scales.cuda(), 256 * 32)).cpu()
    want = torch.from_numpy(ref_values(codes.numpy(), scales.numpy(), 256 * 32)).to(torch.bfloat16)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(back), nan) and torch.equal(back[~nan], want[~nan])


@pytest.mark.gpu
def test_rows_behind_the_last_stay():
    m, k = 5, 392
    X = bf16_randn((m, k), 1.0, torch.Generator().manual_seed(2)).cuda()
    codes = torch.full((m + 2, 16, 32), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((m + 2, 16), 99, dtype=torch.uint8, device="cuda")
    out = torch.full((m + 2, k), 5.0, dtype=torch.bfloat16, device="cuda")
    X8 = lf.lora_mxint8_quantize(X, codes=codes[:m], scales=scales[:m])
    lf.lora_mxint8_dequantize(X8, out=out[:m])
    torch.cuda.synchronize()
    assert (codes[m:] == 99).all() and (scales[m:] == 99).all() and (out[m:] == 5).all()
    assert (X8.codes[:, 13:] == 0).all() and (X8.scales[:, 13:] == 127).all()  # padding


@pytest.mark.gpu
def test_input_past_32_bits():
    # more than 2^31 values: the last rows are the first ones
    m, k = 150000, 14336
    rows = bf16_randn((1000, k), 1.0, torch.Generator().manual_seed(3)).cuda()
    X = rows.repeat(m // 1000, 1)
    X8 = lf.lora_mxint8_quantize(X)
    one = lf.lora_mxint8_quantize(rows)
    assert torch.equal(X8.codes[-1000:], one.codes) and torch.equal(X8.scales[-1000:], one.scales)
    del X
    back = lf.lora_mxint8_dequantize(X8)
    assert torch.equal(back[-1000:], lf.lora_mxint8_dequantize(one))


# ---- the backward (GPU) -----------------------------------------------------------------------------

def weights(k, n, g):
    """The frozen weight in each of its forms."""
    W = bf16_randn((k, n), k ** -0.5, g).cuda()
    return [W, lf.lora_mxfp4_quantize(W), lf.lora_int4_quantize(W, 64)]


def in_bf16(W):
    if isinstance(W, lf.Mxfp4Weight):
        return lf.lora_mxfp4_dequantize(W)
    return lf.lora_int4_dequantize(W) if isinstance(W, lf.Int4Weight) else W


def layer_bwd(W):
    return (lf.lora_mxfp4_linear_bwd if isinstance(W, lf.Mxfp4Weight) else lf.lora_int4_linear_bwd if isinstance(W, lf.Int4Weight)
            else lf.lora_linear_bwd)


BWD = [
    # m, k, n, r, p
    (1, 8, 8, 1, 0.0), (1, 136, 72, 8, 0.1), (5, 264, 136, 5, 0.3), (17, 1032, 264, 16, 0.0), (31, 128, 40, 13, 0.1), (33, 392, 136, 32, 0.2),
    (64, 2056, 72, 64, 0.1), (100, 520, 264, 48, 0.0), (257, 648, 136, 128, 0.1), (300, 264, 520, 100, 0.05), (333, 1032, 776, 5, 0.2),
    (436, 1328, 264, 113, 0.05), (90, 136, 72, 26, 0.0), (129, 264, 136, 127, 0.2), (520, 400, 264, 130, 0.1), (40, 136, 72, 256, 0.0), (1030, 4104, 136, 16, 0.1), (2100, 2048, 72, 12, 0.0), (700, 8192, 40, 64, 0.1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "mxfp4", "int4"])
@pytest.mark.parametrize("at", range(len(BWD)))
def test_backward(at, form):
    m, k, n, r, p = BWD[at]
    log(f"backward m={m} k={k} n={n} r={r} p={p} {form}")
    g = torch.Generator().manual_seed(300 + at)
    W = weights(k, n, g)[["bf16", "mxfp4", "int4"].index(form)]
    X, A, B, dY = (bf16_randn(s, d, g).cuda() for s, d in (((m, k), 1.0), ((k, r), k ** -0.5), ((r, n), 0.02 ** 0.5), ((m, n), 1.0)))
    _, S, keep = lf.lora_linear_fwd(X, in_bf16(W), A, B, 2.0, p, 7, 16)
    X8 = lf.lora_mxint8_quantize(X)
    Xr = lf.lora_mxint8_dequantize(X8)
    dXb = torch.full((m + 3, k), 5.0, dtype=torch.bfloat16, device="cuda")
    dX, dA, dB = lf.lora_mxint8_linear_bwd(dY, X8, W, A, B, S, keep, 2.0, p, dX=dXb[:m])
    rX, rA, rB = layer_bwd(W)(dY, Xr, W, A, B, S, keep, 2.0, p)
    torch.cuda.synchronize()
    assert (dXb[m:] == 5).all()
    if r % 8 == 0:
        assert torch.equal(dA, rA) and torch.equal(dB, rB)
        assert (p > 0 and k % 128) or torch.equal(dX, rX)
    want, slack = layer_reference(X.cpu(), f64(in_bf16(W)), A, B, dY.cpu(), 2.0, p, 7, 16)
    near("dX", dX, want["dX"], slack["dX"])
    near("dB", dB, want["dB"], slack["dB"])
    want, slack = layer_reference(Xr.cpu(), f64(in_bf16(W)), A, B, dY.cpu(), 2.0, p, 7, 16)
    near("dA", dA, want["dA"], slack["dA"])
    none, dA2, dB2 = lf.lora_mxint8_linear_bwd(dY, X8, W, A, B, S, keep, 2.0, p, want_dX=False)
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "mxfp4", "int4"])
@pytest.mark.parametrize("m,k,n,nseg,r_max", [(1, 136, 72, 1, 8), (40, 1032, 264, 7, 16), (100, 264, 136, 60, 40), (600, 520, 136, 5, 128),
                                              (300, 264, 72, 4, 13), (150, 264, 136, 3, 93), (200, 392, 136, 9, 200), (2000, 2056, 72, 6, 64)])
def test_mixed_backward(m, k, n, nseg, r_max, form):
    g = torch.Generator().manual_seed(m + nseg)
    W = weights(k, n, g)[["bf16", "mxfp4", "int4"].index(form)]
    X, dY = bf16_randn((m, k), 1.0, g).cuda(), bf16_randn((m, n), 1.0, g).cuda()
    ranks = [1 + int(torch.randint(0, r_max, (1,), generator=g)) for _ in range(min(nseg, 5))] + [r_max, 3]
    ps = [(0.0, 0.1, 0.3)[i % 3] for i in range(len(ranks))]
    As = [bf16_randn((k, r), k ** -0.5, g).cuda() for r in ranks]
    Bs = [bf16_randn((r, n), 0.02 ** 0.5, g).cuda() for r in ranks]
    cuts = torch.randint(0, m + 1, (nseg - 1,), generator=g).sort().values.tolist()
    seg_off, seg_ad = [0, *cuts, m], torch.randint(0, len(ranks) - 1, (nseg,), generator=g).tolist()
    so = torch.tensor(seg_off, dtype=torch.int64, device="cuda")
    sa = torch.tensor(seg_ad, dtype=torch.int32, device="cuda")
    rm, na = max(ranks), len(ranks)
    plain = lf.adapter_table(As, Bs, [0.5] * na, ps)
    _, S, keep = lf.multi_lora_linear_fwd(X, in_bf16(W), plain, na, so, sa, rm, 3, 8)
    X8 = lf.lora_mxint8_quantize(X)
    Xr = lf.lora_mxint8_dequantize(X8)
    outs = []
    for call, x in ((lf.multi_lora_mxint8_linear_bwd, X8),
                    (lf.multi_lora_mxfp4_linear_bwd if form == "mxfp4" else lf.multi_lora_int4_linear_bwd if form == "int4"
                     else lf.multi_lora_linear_bwd, Xr)):
        dAs, dBs = [torch.full_like(a, 7.0) for a in As], [torch.full_like(b, 7.0) for b in Bs]
        table = lf.adapter_table(As, Bs, [0.5] * na, ps, dAs, dBs)
        dX = call(dY, x, W, table, na, so, sa, S, keep, rm)
        torch.cuda.synchronize()
        outs.append((dX, *dAs, *dBs))
    if rm % 8 == 0:
        for i, (a, b) in enumerate(zip(*outs)):
            assert (i == 0 and k % 128) or torch.equal(a, b), i
    assert not outs[0][na].any()  # the last adapter has no rows
    sums = {}
    for s, a in enumerate(seg_ad):
        lo, hi = seg_off[s], seg_off[s + 1]
        if hi > lo:
            want, slack = layer_reference(X[lo:hi].cpu(), f64(in_bf16(W)), As[a], Bs[a], dY[lo:hi].cpu(), 0.5, ps[a], 3, 8 + lo * k)
            near(f"dX[{s}]", outs[0][0][lo:hi], want["dX"], slack["dX"])
            saved, sslack = layer_reference(Xr[lo:hi].cpu(), f64(in_bf16(W)), As[a], Bs[a], dY[lo:hi].cpu(), 0.5, ps[a], 3, 8 + lo * k)
            for at, w, e in ((1 + a, saved["dA"], sslack["dA"]), (1 + na + a, want["dB"], slack["dB"])):
                # (the other segments' sums are added: their roundings and one more for each segment)
                w0, e0 = sums.get(at, (0.0, 0.0))
                sums[at] = w0 + w, e0 + e + (nseg + 1) * 2.0 ** -24 * np.abs(w)
    for at, (w, e) in sums.items():
        near(f"gradient {at}", outs[0][at], w, e)


@pytest.mark.gpu
@pytest.mark.parametrize("seg_off,seg_ad", [([0, -(1 << 33) + 5, 1 << 40, 20], [0, 1, 0]), ([0, 30, 10, 20], [1, 0, 1]),
                                            ([-7, 4, 4, 1 << 33], [0, 9, -3])])
def test_bad_segment_tables_stay_in_bounds(seg_off, seg_ad):
    m, k, n = 20, 264, 136
    g = torch.Generator().manual_seed(8)
    W = weights(k, n, g)[0]
    As = [bf16_randn((k, r), 1.0, g).cuda() for r in (8, 40)]
    Bs = [bf16_randn((r, n), 1.0, g).cuda() for r in (8, 40)]
    room = [torch.full((t.numel() + 512,), 5.0, dtype=torch.bfloat16, device="cuda") for t in (*As, *Bs)]
    grads = [r[256:256 + t.numel()].view_as(t) for r, t in zip(room, (*As, *Bs))]
    table = lf.adapter_table(As, Bs, [1.0, 2.0], [0.1, 0.0], grads[:2], grads[2:])
    so = torch.tensor(seg_off, dtype=torch.int64, device="cuda")
    sa = torch.tensor(seg_ad, dtype=torch.int32, device="cuda")
    X8 = lf.lora_mxint8_quantize(bf16_randn((m, k), 1.0, g).cuda())
    dX = torch.full((m + 80, k), 5.0, dtype=torch.bfloat16, device="cuda")
    S, keep = torch.zeros(m, 40, device="cuda"), torch.full((m, 9), -1, dtype=torch.int32, device="cuda")
    lf.multi_lora_mxint8_linear_bwd(bf16_randn((m, n), 1.0, g).cuda(), X8, W, table, 2, so, sa, S, keep, 40, dX=dX[40:40 + m])
    torch.cuda.synchronize()
    assert (dX[:40] == 5).all() and (dX[40 + m:] == 5).all()
    assert all((r[:256] == 5).all() and (r[-256:] == 5).all() for r in room)


@pytest.mark.gpu
@pytest.mark.parametrize("r", [8, 13])
def test_marked_blocks_reach_their_columns_only(r):
    # a NaN block of the saved input makes its rows of dA NaN (the columns of X it holds), and nothing else
    m, k, n = 70, 392, 72
    g = torch.Generator().manual_seed(5)
    W = weights(k, n, g)[0]
    X, A, B, dY = (bf16_randn(s, 1.0, g).cuda() for s in ((m, k), (k, r), (r, n), (m, n)))
    _, S, keep = lf.lora_linear_fwd(X, W, A, B, 2.0, 0.0)
    want = lf.lora_mxint8_linear_bwd(dY, lf.lora_mxint8_quantize(X), W, A, B, S, keep, 2.0, 0.0)
    X[33, 70] = float("inf")
    got = lf.lora_mxint8_linear_bwd(dY, lf.lora_mxint8_quantize(X), W, A, B, S, keep, 2.0, 0.0)
    bad = torch.zeros(k, dtype=torch.bool, device="cuda")
    bad[64:96] = True
    assert torch.isnan(got[1][bad]).all() and torch.equal(got[1][~bad], want[1][~bad])
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


@pytest.mark.gpu
@pytest.mark.parametrize("m,r", [(33, 9), (300, 40)])
def test_unaligned_adapter_gives_the_same(m, r):
    k, n = 264, 136
    g = torch.Generator().manual_seed(31)
    W = weights(k, n, g)[2]
    X, A, B, dY = (bf16_randn(s, d, g) for s, d in (((m, k), 1.0), ((k, r), k ** -0.5), ((r, n), 0.1), ((m, n), 1.0)))
    A1, B1, dY, X8 = offset_view(A), offset_view(B), dY.cuda(), lf.lora_mxint8_quantize(X.cuda())
    _, S, keep = lf.lora_linear_fwd(X.cuda(), in_bf16(W), A1, B1, 2.0, 0.1, 3, 0)
    a = lf.lora_mxint8_linear_bwd(dY, X8, W, A1, B1, S, keep, 2.0, 0.1)
    b = lf.lora_mxint8_linear_bwd(dY, X8, W, A.cuda(), B.cuda(), S, keep, 2.0, 0.1)
    want, slack = layer_reference(X, f64(in_bf16(W)), A, B, dY.cpu(), 2.0, 0.1, 3, 0)  # (dB is of the forward's S)
    saved, sslack = layer_reference(lf.lora_mxint8_dequantize(X8).cpu(), f64(in_bf16(W)), A, B, dY.cpu(), 2.0, 0.1, 3, 0)
    for dX, dA, dB in (a, b):
        near("dX", dX, want["dX"], slack["dX"])
        near("dA", dA, saved["dA"], sslack["dA"])
        near("dB", dB, want["dB"], slack["dB"])


@pytest.mark.gpu
@pytest.mark.parametrize("r", [8, 5, 130])
def test_no_rows(r):
    k, n = 136, 72
    g = torch.Generator().manual_seed(1)
    A, B = bf16_randn((k, r), 1.0, g).cuda(), bf16_randn((r, n), 1.0, g).cuda()
    for W in weights(k, n, g):
        X8 = lf.lora_mxint8_quantize(torch.empty(0, k, dtype=torch.bfloat16, device="cuda"))
        assert lf.lora_mxint8_dequantize(X8).shape == (0, k)
        dY, S = torch.empty(0, n, dtype=torch.bfloat16, device="cuda"), torch.empty(0, r, device="cuda")
        dX, dA, dB = lf.lora_mxint8_linear_bwd(dY, X8, W, A, B, S, None, 2.0, 0.0)
        torch.cuda.synchronize()
        assert dX.shape == (0, k) and not dA.any() and not dB.any()


# ---- use: streams, graphs, autograd ---------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("m,r,p", [(5, 16, 0.1), (333, 5, 0.1), (700, 64, 0.0)])
@pytest.mark.parametrize("form", [0, 2])
def test_captured_step_replays_match_eager(form, m, r, p):
    k, n = 520, 264
    g = torch.Generator().manual_seed(5)
    W = weights(k, n, g)[form]
    forward = lf.lora_int4_linear_fwd if form else lf.lora_linear_fwd
    X, A, B, dY = (bf16_randn(s, 1.0, g).cuda() for s in ((m, k), (k, r), (r, n), (m, n)))

    def run():
        Y, S, keep = forward(X, W, A, B, 2.0, p, 9, 0)
        X8 = lf.lora_mxint8_quantize(X)
        return (Y, *X8[:2], lf.lora_mxint8_dequantize(X8), *lf.lora_mxint8_linear_bwd(dY, X8, W, A, B, S, keep, 2.0, p))

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
    m, k, n, r = 300, 520, 264, 16
    g = torch.Generator().manual_seed(6)
    W = weights(k, n, g)[0]
    A, B = bf16_randn((k, r), 1.0, g).cuda(), bf16_randn((r, n), 1.0, g).cuda()
    sides = []
    for _ in range(2):
        X, dY = bf16_randn((m, k), 1.0, g).cuda(), bf16_randn((m, n), 1.0, g).cuda()
        _, S, keep = lf.lora_linear_fwd(X, W, A, B, 2.0, 0.1)
        X8 = lf.lora_mxint8_quantize(X)
        sides.append((torch.cuda.Stream(), X, dY, X8, S, keep, lf.lora_mxint8_linear_bwd(dY, X8, W, A, B, S, keep, 2.0, 0.1)))
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for st, X, dY, _, S, keep, want in sides:
            X8 = lf.lora_mxint8_quantize(X, stream=st)
            got.append((lf.lora_mxint8_linear_bwd(dY, X8, W, A, B, S, keep, 2.0, 0.1, stream=st), want, X8))
    torch.cuda.synchronize()
    for a, b, _ in got:
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_autograd_keeps_the_saved_input_alone():
    m, k, n, r = 300, 264, 136, 16
    g = torch.Generator().manual_seed(12)
    W = weights(k, n, g)[0]
    A, B = bf16_randn((k, r), k ** -0.5, g).cuda().requires_grad_(), bf16_randn((r, n), 0.1, g).cuda().requires_grad_()
    X, dY = bf16_randn((m, k), 1.0, g).cuda(), bf16_randn((m, n), 1.0, g).cuda()
    held = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: held.append(t) or t, lambda t: t):
        x = X.clone().requires_grad_()
        X8 = lf.lora_mxint8_quantize(X)
        Y = lf.lora_linear(x.view(3, 100, k), W, A, B, 2.0, 0.1, 11, 8, X8=X8)
    assert not any(t.dtype == torch.bfloat16 and t.numel() == m * k for t in held)
    assert any(t.data_ptr() == X8.codes.data_ptr() for t in held)
    Y.backward(dY.view(3, 100, n))
    want, slack = layer_reference(X.cpu(), f64(W), A, B, dY.cpu(), 2.0, 0.1, 11, 8)
    saved, sslack = layer_reference(lf.lora_mxint8_dequantize(X8).cpu(), f64(W), A, B, dY.cpu(), 2.0, 0.1, 11, 8)
    near("Y", Y.reshape(m, n), want["Y"], slack["Y"])
    near("dX", x.grad, want["dX"], slack["dX"])
    near("dB", B.grad, want["dB"], slack["dB"])
    near("dA", A.grad, saved["dA"], sslack["dA"])
    # against the gradient of the exact input: each X' is off by 2^-7 of its block's largest value at most
    off = np.abs(f64(X8.codes) * 0 + 0.5) * 2.0 ** (f64(X8.scales)[..., None] - 127)
    off = off.reshape(m, -1)[:, :k] / 0.9
    dS = 2.0 * f64(dY) @ f64(B).T
    assert (np.abs(saved["dA"] - want["dA"]) <= off.T @ np.abs(dS) * 1.001).all()


@pytest.mark.gpu
def test_modules_share_a_saved_input():
    m, k, n, r = 90, 264, 136, 8
    g = torch.Generator().manual_seed(13)
    layers = [lf.LoraLinear(W, r, 2.0, 0.0, seed=i, save_bits=8) for i, W in enumerate(weights(k, n, g))]
    for l in layers:
        with torch.no_grad():
            l.B.copy_(bf16_randn((r, n), 0.1, g))
    X = bf16_randn((m, k), 1.0, g).cuda()

    def grads(X8):
        for l in layers:
            l.A.grad = l.B.grad = None
        x = X.clone().requires_grad_()
        sum(l(x, X8).float().square().sum() for l in layers).backward()
        return [x.grad] + [t.grad for l in layers for t in (l.A, l.B)]

    own, shared = grads(None), grads(lf.lora_mxint8_quantize(X))
    assert all(torch.equal(a, b) for a, b in zip(own, shared))
    with torch.no_grad():
        assert torch.equal(layers[0](X), layers[0](X))
    for l in layers:
        l.save_bits = 16
    full = grads(None)
    assert torch.equal(full[0], own[0]) and all(torch.equal(a, b) for a, b in zip(full[2::2], own[2::2]))  # dX, dB
    gc.collect()


@pytest.mark.gpu
def test_mixed_autograd_and_optimizer_run():
    # a step as it is used: the 4-bit weight, the input in 8 bits, two adapters, AdamW; then single tokens
    m, k, n, ranks = 96, 264, 136, [16, 8]
    g = torch.Generator().manual_seed(2)
    W = weights(k, n, g)[2]
    As = [bf16_randn((k, r), k ** -0.5, g).cuda().requires_grad_() for r in ranks]
    Bs = [bf16_randn((r, n), 0.02 ** 0.5, g).cuda().requires_grad_() for r in ranks]
    so = torch.tensor([0, 40, m], dtype=torch.int64, device="cuda")
    sa = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    opt = lf.LoraAdamW([*As, *Bs], lr=1e-3)
    X, dY = bf16_randn((m, k), 1.0, g).cuda(), bf16_randn((m, n), 1.0, g).cuda()
    for step in range(2):
        before = [t.detach().clone() for t in (*As, *Bs)]
        x = X.clone().requires_grad_()
        X8 = lf.lora_mxint8_quantize(X)
        Y = lf.multi_lora_linear(x, W, so, sa, As, Bs, [2.0, 1.0], [0.1, 0.0], 3, 16 + step * m * k, X8=X8)
        Y.backward(dY)
        Xr, Wr = lf.lora_mxint8_dequantize(X8).cpu(), f64(in_bf16(W))
        for lo, hi, a, alpha, p in ((0, 40, 1, 1.0, 0.0), (40, m, 0, 2.0, 0.1)):
            at = 16 + step * m * k + lo * k
            want, slack = layer_reference(X[lo:hi].cpu(), Wr, As[a], Bs[a], dY[lo:hi].cpu(), alpha, p, 3, at)
            saved, sslack = layer_reference(Xr[lo:hi], Wr, As[a], Bs[a], dY[lo:hi].cpu(), alpha, p, 3, at)
            near("dX", x.grad[lo:hi], want["dX"], slack["dX"])
            near("dA", As[a].grad, saved["dA"], sslack["dA"])
            near("dB", Bs[a].grad, want["dB"], slack["dB"])
        opt.step()
        opt.zero_grad()
        assert all(not torch.equal(a, b) for a, b in zip(before, (*As, *Bs)))
    with torch.no_grad():
        tokens = bf16_randn((2, k), 1.0, g).cuda()
        one = torch.tensor([0, 1, 2], dtype=torch.int64, device="cuda")
        Y = lf.multi_lora_linear(tokens, W, one, sa, As, Bs, [2.0, 1.0], [0.0, 0.0])
        for i, a in enumerate((1, 0)):
            alone = lf.lora_linear(tokens[i:i + 1], W, As[a], Bs[a], [2.0, 1.0][a])
            x, w = f64(tokens[i:i + 1]), f64(in_bf16(W))
            # (the weight may be rounded or not, and each result is rounded: two half steps and the sums')
            mag = np.abs(x) @ np.abs(w)
            assert (np.abs(f64(Y[i:i + 1]) - f64(alone)) <= 2.0 ** -7 * np.abs(f64(alone)) + 2.0 ** -7 * mag).all()
