"""A layer's input saved in 8 bits (MXINT8), and the layer's backward from it.

Every function has the name of a C-ABI entry point in include/lora_fused.h and
only marshals arguments, as the rest of the binding does.  `lora_linear` and
`multi_lora_linear` take a saved input (X8) for their backward; `LoraLinear`
makes one itself with save_bits=8.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import int4, mxfp4
from ._lib import _check, _elsewhere, _handle, _need, _need_on, _on_device, _scratch, load
from .int4 import Int4Weight, _matrix, _need_segments, _out, _sizes
from .mxfp4 import Mxfp4Weight

_BF16, _F32 = torch.bfloat16, torch.float32
KIND_BF16, KIND_MXFP4, KIND_INT4 = 0, 1, 2


class Mxint8Input(NamedTuple):
    """An m x k input as 8-bit integers and power-of-two scales, one scale for
    32 values of a row: value (i, 32 b + j) is codes[i, b, j] *
    2^(scales[i, b] - 127).  `codes` (m, 4 ceil(k/128), 32) int8 and `scales`
    (m, 4 ceil(k/128)) uint8 are device tensors."""
    codes: torch.Tensor
    scales: torch.Tensor
    k: int

    @property
    def shape(self):
        return (self.codes.shape[0], self.k)

    @property
    def device(self):
        return self.codes.device


def _need_input(X8: Mxint8Input):
    if not isinstance(X8, Mxint8Input):
        raise TypeError(f"X8 must be an Mxint8Input, got {type(X8).__name__}")
    codes, scales, k = X8
    blocks = (k + 127) // 128 * 4
    m = codes.shape[0] if codes.dim() == 3 else -1
    if codes.shape != (m, blocks, 32) or scales.shape != (m, blocks):
        raise ValueError(f"X8.codes {tuple(codes.shape)} and X8.scales {tuple(scales.shape)} do not hold rows of {k} "
                         f"values ((m, {blocks}, 32) and (m, {blocks}) do)")
    _need(codes, torch.int8, "X8.codes")
    _need_on(scales, scales.shape, torch.uint8, "X8.scales", codes.device)
    return codes, scales, m, k, codes.device


def lora_mxint8_quantize(X, *, codes=None, scales=None, stream=None) -> Mxint8Input:
    """X (m x k bf16) in 8 bits."""
    _need(X, _BF16, "X")
    m, k = _matrix(X, "X")
    dev = X.device
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_mxint8_quantize(X, codes=codes, scales=scales)
    blocks = (k + 127) // 128 * 4
    codes = _out(codes, (m, blocks, 32), torch.int8, "codes", dev)
    scales = _out(scales, (m, blocks), torch.uint8, "scales", dev)
    _check(load().lora_mxint8_quantize(X.data_ptr(), m, k, codes.data_ptr(), scales.data_ptr(), _handle(dev)))
    return Mxint8Input(codes, scales, k)


def lora_mxint8_dequantize(X8: Mxint8Input, *, out=None, stream=None):
    """The m x k bf16 input that X8 stands for (exact)."""
    codes, scales, m, k, dev = _need_input(X8)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_mxint8_dequantize(X8, out=out)
    out = _out(out, (m, k), _BF16, "out", dev)
    _check(load().lora_mxint8_dequantize(codes.data_ptr(), scales.data_ptr(), m, k, out.data_ptr(), _handle(dev)))
    return out


def _weight(W, k: int, dev):
    """(kind, data pointer, scales pointer, group, n) of a frozen weight in any of its forms."""
    if isinstance(W, Mxfp4Weight):
        codes, scales, wk, n, wdev = mxfp4._need_weight(W)
        found = KIND_MXFP4, codes.data_ptr(), scales.data_ptr(), 0, n
    elif isinstance(W, Int4Weight):
        codes, scales, wk, n, group, wdev = int4._need_weight(W)
        found = KIND_INT4, codes.data_ptr(), scales.data_ptr(), group, n
    else:
        _need(W, _BF16, "W")
        (wk, n), wdev = _matrix(W, "W"), W.device
        found = KIND_BF16, W.data_ptr(), None, 0, n
    if wk != k:
        raise ValueError(f"W is {wk} x {n}, the saved input has rows of {k}")
    if wdev != dev:
        raise ValueError(f"W is on {wdev}, the saved input on {dev}")
    return found


@_sizes
def lora_mxint8_linear_bwd_workspace_size(kind, group, m, k, n, r) -> int:
    return load().lora_mxint8_linear_bwd_workspace_size(kind, group, m, k, n, r)


@_sizes
def multi_lora_mxint8_bwd_workspace_size(kind, group, m, k, n, r_max, num_adapters, num_segments) -> int:
    return load().multi_lora_mxint8_bwd_workspace_size(kind, group, m, k, n, r_max, num_adapters, num_segments)


def lora_mxint8_linear_bwd(dY, X8: Mxint8Input, W, A, B, S, keep_bits, alpha: float, p: float, *, dX=None, dA=None,
                           dB=None, workspace=None, stream=None, want_dX: bool = True):
    """lora_linear_bwd from a saved input, over W (bf16, an Mxfp4Weight or an
    Int4Weight).  Returns (dX, dA, dB); dX is None (and its product skipped)
    when want_dX is False."""
    codes, scales, m, k, dev = _need_input(X8)
    kind, data, w_scales, group, n = _weight(W, k, dev)
    r = _matrix(A, "A")[1]
    _need_on(dY, (m, n), _BF16, "dY", dev)
    _need_on(A, (k, r), _BF16, "A", dev)
    _need_on(B, (r, n), _BF16, "B", dev)
    _need_on(S, (m, r), _F32, "S", dev)
    if keep_bits is not None:
        _need_on(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_mxint8_linear_bwd(dY, X8, W, A, B, S, keep_bits, alpha, p, dX=dX, dA=dA, dB=dB,
                                          workspace=workspace, want_dX=want_dX)
    dX = _out(dX, (m, k), _BF16, "dX", dev) if want_dX else None
    dA = _out(dA, (k, r), _BF16, "dA", dev)
    dB = _out(dB, (r, n), _BF16, "dB", dev)
    ws, nb, _held = _scratch(lora_mxint8_linear_bwd_workspace_size(kind, group, m, k, n, r), dev, workspace)
    _check(load().lora_mxint8_linear_bwd(dY.data_ptr(), codes.data_ptr(), scales.data_ptr(), kind, data, w_scales, group,
                                         A.data_ptr(), B.data_ptr(), S.data_ptr(),
                                         None if keep_bits is None else keep_bits.data_ptr(), m, k, n, r, alpha, p,
                                         None if dX is None else dX.data_ptr(), dA.data_ptr(), dB.data_ptr(), ws, nb,
                                         _handle(dev)))
    return dX, dA, dB


def multi_lora_mxint8_linear_bwd(dY, X8: Mxint8Input, W, adapters: torch.Tensor, num_adapters: int, seg_off,
                                 seg_adapter, S, keep_bits, r_max: int, *, dX=None, workspace=None, stream=None,
                                 want_dX: bool = True) -> Optional[torch.Tensor]:
    """multi_lora_linear_bwd from a saved input, over W (bf16, an Mxfp4Weight or
    an Int4Weight): writes the table's dA and dB, returns dX (None, its product
    skipped, when want_dX is False)."""
    codes, scales, m, k, dev = _need_input(X8)
    kind, data, w_scales, group, n = _weight(W, k, dev)
    nseg = _need_segments(seg_off, seg_adapter, adapters, num_adapters, k, n, r_max, dev)
    _need_on(dY, (m, n), _BF16, "dY", dev)
    _need_on(S, (m, r_max), _F32, "S", dev)
    _need_on(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return multi_lora_mxint8_linear_bwd(dY, X8, W, adapters, num_adapters, seg_off, seg_adapter, S, keep_bits,
                                                r_max, dX=dX, workspace=workspace, want_dX=want_dX)
    dX = _out(dX, (m, k), _BF16, "dX", dev) if want_dX else None
    ws, nb, _held = _scratch(multi_lora_mxint8_bwd_workspace_size(kind, group, m, k, n, r_max, num_adapters, nseg), dev,
                             workspace)
    _check(load().multi_lora_mxint8_linear_bwd(dY.data_ptr(), codes.data_ptr(), scales.data_ptr(), kind, data, w_scales,
                                               group, adapters.data_ptr(), num_adapters, seg_off.data_ptr(),
                                               seg_adapter.data_ptr(), nseg, S.data_ptr(), keep_bits.data_ptr(), m, k,
                                               n, r_max, None if dX is None else dX.data_ptr(), ws, nb, _handle(dev)))
    return dX
