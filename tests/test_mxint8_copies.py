"""The copies that the backward from a saved input makes before it: made where something reads them only.

References and tolerances are test_mxint8.py's."""
import pytest
import torch

import lora_fine_tuning_amd as lf
from parity import bf16_randn, log
from test_mxint8 import weights


@pytest.mark.gpu
@pytest.mark.parametrize("form", [0, 1, 2])
@pytest.mark.parametrize("m,k,n,r,p", [(33, 264, 136, 5, 0.2), (300, 1032, 72, 13, 0.0), (70, 128, 72, 121, 0.1)])
def test_adapter_is_copied_for_dx_alone(m, k, n, r, p, form):
    # an odd rank's A is copied with longer rows for the dX product: without dX its place in the workspace,
    # past S's copy, stays as it was
    log(f"copies m={m} k={k} n={n} r={r} form {form}")
    g = torch.Generator().manual_seed(r)
    W = weights(k, n, g)[form]
    X, A, B, dY = (bf16_randn(s, d, g).cuda() for s, d in (((m, k), 1.0), ((k, r), k ** -0.5), ((r, n), 0.1), ((m, n), 1.0)))
    _, S, keep = lf.lora_linear_fwd(X, weights(k, n, torch.Generator().manual_seed(r))[0], A, B, 2.0, p, 7, 16)
    X8 = lf.lora_mxint8_quantize(X)
    group = W.group if form == 2 else 0
    need = lf.lora_mxint8_linear_bwd_workspace_size(form, group, m, k, n, r)
    row, up = -(-r // 8) * 8, lambda v: -(-v // 256) * 256
    at, size = up(m * row * 4), k * row * 2
    place = torch.zeros(k, row, dtype=torch.bfloat16, device="cuda")
    place[:, :r] = A
    outs = []
    for want in (False, True):
        room = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
        outs.append(lf.lora_mxint8_linear_bwd(dY, X8, W, A, B, S, keep, 2.0, p, workspace=room, want_dX=want))
        torch.cuda.synchronize()
        held = room[at:at + size]
        if want:
            assert torch.equal(held, place.view(torch.uint8).flatten())
        else:
            assert (held == 0x5A).all()
    assert outs[0][0] is None and torch.equal(outs[0][1], outs[1][1]) and torch.equal(outs[0][2], outs[1][2])
