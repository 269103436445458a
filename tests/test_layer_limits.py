"""Sizes at and past what the layer's calls address with 32 bits: refused on the host, with nothing enqueued.

No kernel is launched: the pointers are fake, and every call here is refused."""
import os

import pytest
import torch

import lora_fine_tuning_amd as lf
from lora_fine_tuning_amd import _lib

FAKE = 0x10000  # aligned, never dereferenced
UNSUPPORTED, WORKSPACE = -2, -3
BF16, MXFP4, INT4 = 0, 1, 2
F, BIG = FAKE, 1 << 62


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("host-only checks; a GPU is visible")
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    return _lib.load()


def backwards(lib, m, k, n, r, wsb=BIG):
    """Every backward call of the layer at a size, by name."""
    tail = (F, F, F, F, wsb, None)  # dX, dA, dB, the workspace
    multi = (F, F, wsb, None)
    yield "bf16", lib.lora_linear_bwd(F, F, F, F, F, F, F, m, k, n, r, 1.0, 0.1, *tail)
    yield "bf16 noalloc", lib.lora_linear_bwd_noalloc(F, F, F, F, F, F, F, m, k, n, r, 1.0, 0.1, F, F, F, None)
    yield "bf16 mixed", lib.multi_lora_linear_bwd(F, F, F, F, 2, F, F, 1, F, F, m, k, n, r, *multi)
    yield "mxfp4", lib.lora_mxfp4_linear_bwd(F, F, F, F, F, F, F, F, m, k, n, r, 1.0, 0.1, *tail)
    yield "mxfp4 mixed", lib.multi_lora_mxfp4_linear_bwd(F, F, F, F, F, 2, F, F, 1, F, F, m, k, n, r, *multi)
    yield "int4", lib.lora_int4_linear_bwd(F, F, F, F, 64, F, F, F, F, m, k, n, r, 1.0, 0.1, *tail)
    yield "int4 mixed", lib.multi_lora_int4_linear_bwd(F, F, F, F, 64, F, 2, F, F, 1, F, F, m, k, n, r, *multi)
    yield from saved_backwards(lib, m, k, n, r, wsb)


def saved_backwards(lib, m, k, n, r, wsb=BIG):
    for kind in (BF16, MXFP4, INT4):
        yield f"saved {kind}", lib.lora_mxint8_linear_bwd(F, F, F, kind, F, F, 64, F, F, F, F, m, k, n, r, 1.0, 0.1, F, F, F, F, wsb, None)
        yield f"saved {kind} mixed", lib.multi_lora_mxint8_linear_bwd(F, F, F, kind, F, F, 64, F, 2, F, F, 1, F, F, m, k, n, r, F, F, wsb, None)


def queries(m, k, n, r):
    yield _lib.lora_linear_bwd_workspace_size(m, k, n, r)
    yield _lib.multi_lora_bwd_workspace_size(m, k, n, r, 2, 1)
    yield lf.lora_mxfp4_linear_bwd_workspace_size(m, k, n, r)
    yield lf.multi_lora_mxfp4_bwd_workspace_size(m, k, n, r, 2, 1)
    yield lf.lora_int4_linear_bwd_workspace_size(m, k, n, 64, r)
    yield lf.multi_lora_int4_bwd_workspace_size(m, k, n, 64, r, 2, 1)
    for kind in (BF16, MXFP4, INT4):
        yield lf.lora_mxint8_linear_bwd_workspace_size(kind, 64, m, k, n, r)
        yield lf.multi_lora_mxint8_bwd_workspace_size(kind, 64, m, k, n, r, 2, 1)


@pytest.mark.parametrize("m", [0, 1, 100])
@pytest.mark.parametrize("k", [1 << 25, (1 << 25) + 8, 1 << 26])
def test_backward_of_too_long_rows(lib, m, k):
    # (the plan divided by a row count of zero here, which ended the process)
    assert all(q == 0 for q in queries(m, k, 8, 8))
    for name, status in backwards(lib, m, k, 8, 8):
        assert status == UNSUPPORTED, name


def test_backward_of_the_longest_rows(lib):
    k = (1 << 25) - 8
    assert all(q > 0 for q in queries(4, k, 8, 8))
    for name, status in backwards(lib, 4, k, 8, 8, wsb=0):
        assert status == (UNSUPPORTED if name == "bf16 noalloc" else WORKSPACE), name


@pytest.mark.parametrize("kind", [BF16, MXFP4, INT4])
def test_saved_input_counts_the_widened_adapter(lib, kind):
    # the dX product reads A with its ranks rounded up to 8: 57 x 2^24 bf16 is under 2 GiB, 64 x 2^24 is not
    def status(k, r, dX, wsb=0):
        return lib.lora_mxint8_linear_bwd(F, F, F, kind, F, F, 64, F, F, F, F, 4, k, 8, r, 1.0, 0.1, dX, F, F, F, wsb, None)

    for k, r in ((1 << 24, 57), (1 << 24, 63), (1 << 23, 121), (1 << 22, 249)):
        assert r * k * 2 < 1 << 31
        assert status(k, r, F, BIG) == UNSUPPORTED
        assert status(k, r, None) == WORKSPACE  # (without dX nothing reads A)
        assert status(k - 8, r, F) == WORKSPACE


@pytest.mark.parametrize("m", [1, 64])
def test_four_bit_forward_expands_past_its_limits_alone(m):
    # up to 64 rows the packed weight is read for k <= 2^20 and n <= 2^24; past them there is room for W' in bf16
    for k, n, expands in ((1 << 20, 16, False), ((1 << 20) + 8, 16, True), (16, 1 << 24, False), (16, (1 << 24) + 8, True)):
        for need in (lf.lora_int4_frozen_fwd_workspace_size(m, k, n, 64), lf.lora_int4_linear_fwd_workspace_size(m, k, n, 64, 8)):
            part = 16 * m * n * 4 + 4 * (k // 1024 + 1) * m * 8  # the most that slices and S's partial sums take
            assert need >= 2 * k * n if expands else need <= part + (1 << 20), (k, n)


@pytest.mark.parametrize("kind", [-1, 3, 7])
def test_saved_input_query_of_an_unknown_weight(kind):
    for r in (5, 8, 200):
        assert lf.lora_mxint8_linear_bwd_workspace_size(kind, 64, 100, 264, 136, r) == 0
        assert lf.multi_lora_mxint8_bwd_workspace_size(kind, 64, 100, 264, 136, r, 2, 1) == 0


def forwards(lib, m, k, n, r=8, wsb=BIG):
    tail = (F, F, F, F, wsb, None)  # Y, S, the mask, the workspace
    yield "bf16 frozen", lib.lora_frozen_fwd(F, F, m, k, n, F, None)
    yield "bf16", lib.lora_linear_fwd(F, F, F, F, m, k, n, r, 1.0, 0.1, 0, 0, *tail)
    yield "bf16 concat", lib.lora_linear_fwd_concat(F, F, F, F, m, k, n, r, 1.0, F, F, None)
    yield "bf16 mixed", lib.multi_lora_linear_fwd(F, F, F, 2, F, F, 1, m, k, n, r, 0, 0, *tail)
    yield "mxfp4 frozen", lib.lora_mxfp4_frozen_fwd(F, F, F, m, k, n, F, F, wsb, None)
    yield "mxfp4", lib.lora_mxfp4_linear_fwd(F, F, F, F, F, m, k, n, r, 1.0, 0.1, 0, 0, *tail)
    yield "mxfp4 mixed", lib.multi_lora_mxfp4_linear_fwd(F, F, F, F, 2, F, F, 1, m, k, n, r, 0, 0, *tail)
    yield "int4 frozen", lib.lora_int4_frozen_fwd(F, F, F, 64, m, k, n, F, F, wsb, None)
    yield "int4", lib.lora_int4_linear_fwd(F, F, F, 64, F, F, m, k, n, r, 1.0, 0.1, 0, 0, *tail)
    yield "int4 mixed", lib.multi_lora_int4_linear_fwd(F, F, F, 64, F, 2, F, F, 1, m, k, n, r, 0, 0, *tail)


def frozen_backwards(lib, m, k, n, wsb=BIG):
    yield "bf16 frozen", lib.lora_frozen_bwd(F, F, m, k, n, F, None)
    yield "mxfp4 frozen", lib.lora_mxfp4_frozen_bwd(F, F, F, m, k, n, F, F, wsb, None)
    yield "int4 frozen", lib.lora_int4_frozen_bwd(F, F, F, 64, m, k, n, F, F, wsb, None)


@pytest.mark.parametrize("m,k,n", [(256, 1 << 22, 8), (1000, 1 << 22, 64), (100, 11 << 20, 8), (1, 64, (1 << 24) + 8), (256, 8, (1 << 24) + 8)])
def test_forward_of_tiles_past_two_gigabytes(lib, m, k, n):
    # (rows of a tile past 2^31 bytes were read as zeros, or as others past 2^32, and their outputs dropped)
    for name, status in forwards(lib, m, k, n):
        assert status == UNSUPPORTED, name


@pytest.mark.parametrize("m,k,n", [(256, 8, 1 << 22), (300, 1 << 22, 8), (100, 11 << 20, 8), (8, 8, 1 << 27), (1, 256, 1 << 22)])
def test_backward_of_tiles_past_two_gigabytes(lib, m, k, n):
    for name, status in (*backwards(lib, m, k, n, 7), *frozen_backwards(lib, m, k, n)):
        assert status == UNSUPPORTED, name


def test_tiles_of_just_two_gigabytes(lib):
    for m, k, n in ((255, 1 << 22, 8), (256, (1 << 22) - 8, 8), (1, 64, (1 << 24) - 8), (1, 1 << 24, 8)):
        for name, status in forwards(lib, m, k, n, wsb=0):
            assert status != UNSUPPORTED, name
    for m, k, n in ((255, 8, 1 << 22), (256, 8, (1 << 22) - 8), (1, 248, 1 << 22), (7, 8, (1 << 27) - 8)):
        for name, status in (*backwards(lib, m, k, n, 7, wsb=0), *frozen_backwards(lib, m, k, n, wsb=0)):
            assert status != UNSUPPORTED or "noalloc" in name, name
    # no dX: no product over W
    assert lib.lora_linear_bwd(F, F, F, F, F, F, F, 256, 8, 1 << 22, 7, 1.0, 0.1, None, F, F, F, 0, None) == WORKSPACE
