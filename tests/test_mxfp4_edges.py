"""Calls over an MXFP4 weight that the documentation allows and that reach further than the
layers' own tests: segment tables with any content.

The references and tolerances are those of test_mxfp4.py."""
import pytest
import torch

import lora_fine_tuning_amd as lf
from parity import bf16_randn, log
from test_mxfp4 import layer_case, layer_reference, near

LAST = (1 << 63) - 1


def mixed_set(k, n, ranks, alphas, ps, seed):
    """(table, As, Bs, dAs, dBs): a table holds addresses only, so its tensors come along."""
    g = torch.Generator().manual_seed(seed)
    As = [bf16_randn((k, r), k ** -0.5, g).cuda() for r in ranks]
    Bs = [bf16_randn((r, n), 0.02 ** 0.5, g).cuda() for r in ranks]
    dAs, dBs = [torch.zeros_like(a) for a in As], [torch.zeros_like(b) for b in Bs]
    return lf.adapter_table(As, Bs, alphas, ps, dAs, dBs), As, Bs, dAs, dBs


@pytest.mark.gpu
@pytest.mark.parametrize("m", [20, 100])
@pytest.mark.parametrize("ends", [[LAST, LAST, LAST], [LAST - 40, LAST, 100], [-LAST - 1, LAST, -LAST - 1]])
def test_segment_offsets_may_be_any_number(m, ends):
    # an end past the last row stands for it, and a segment that begins there has no rows, whatever is added
    # to its offset; nothing outside the buffers is written
    k, n = 1032, 136
    log(f"m={m} ends={ends}")
    X, W4, W, _, _, dY = layer_case(m, k, n, 8, seed=m)
    table, As, Bs, *_ = mixed_set(k, n, (8, 40), [1.0, 2.0], [0.1, 0.0], seed=8)
    so = torch.tensor([0, 10, *ends], dtype=torch.int64, device="cuda")
    sa = torch.tensor([0, 1, 0, 1], dtype=torch.int32, device="cuda")
    Y = torch.full((m + 80, n), 5.0, dtype=torch.bfloat16, device="cuda")
    S = torch.full((m + 80, 40), 5.0, device="cuda")
    keep = torch.full((m + 80, (k + 31) // 32), 5, dtype=torch.int32, device="cuda")
    mid = slice(40, 40 + m)
    lf.multi_lora_mxfp4_linear_fwd(X.cuda(), W4, table, 2, so, sa, 40, 3, 8, Y=Y[mid], S=S[mid], keep_bits=keep[mid])
    torch.cuda.synchronize()
    for t in (Y, S, keep):
        assert (t[:40] == 5).all() and (t[40 + m:] == 5).all()
    want, slack = layer_reference(X[:10], W, As[0].cpu(), Bs[0].cpu(), dY[:10], 1.0, 0.1, 3, 8)
    near("Y", Y[40:50], want["Y"], slack["Y"])
    if ends[0] > 0:
        want, slack = layer_reference(X[10:], W, As[1].cpu(), Bs[1].cpu(), dY[10:], 2.0, 0.0, 3, 8 + 10 * k)
        near("Y", Y[50:40 + m], want["Y"], slack["Y"])
