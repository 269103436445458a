"""Frozen weights held in 4 bits (MXFP4) and the layers over them.

Every function has the name of a C-ABI entry point in include/lora_fused.h and
only marshals arguments, as the rest of the binding does.  `lora_linear`,
`multi_lora_linear` and `LoraLinear` take an Mxfp4Weight wherever they take W.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch

from ._lib import (_check, _check_table, _elsewhere, _handle, _need, _need_on, _on_device, _scratch, load)

_BF16, _F32 = torch.bfloat16, torch.float32
_sizes = functools.lru_cache(maxsize=1024)  # a workspace's size follows from the sizes asked for alone


class Mxfp4Weight(NamedTuple):
    """A frozen k x n weight as e2m1 codes and power-of-two scales, one scale
    for 32 rows of a column.  `codes` (ceil(n/16), 4 ceil(k/128), 16, 16) and
    `scales` (ceil(n/16), 4 ceil(k/128), 16) are uint8 device tensors; byte i
    of codes[c, b, j] holds rows 32 b + 2 i (low nibble) and 32 b + 2 i + 1 of
    column 16 c + j."""
    codes: torch.Tensor
    scales: torch.Tensor
    k: int
    n: int

    @property
    def shape(self):
        return (self.k, self.n)

    @property
    def device(self):
        return self.codes.device


def _need_weight(W: Mxfp4Weight):
    if not isinstance(W, Mxfp4Weight):
        raise TypeError(f"W must be an Mxfp4Weight, got {type(W).__name__}")
    codes, scales, k, n = W
    groups, blocks = (n + 15) // 16, (k + 127) // 128 * 4
    if (codes.shape == (groups, blocks, 16, 16) and scales.shape == (groups, blocks, 16) and codes.is_cuda
            and codes.dtype is torch.uint8 and scales.dtype is torch.uint8 and codes.is_contiguous()
            and scales.is_contiguous() and scales.get_device() == codes.get_device()):
        return codes, scales, k, n, codes.device
    if codes.shape != (groups, blocks, 16, 16) or scales.shape != (groups, blocks, 16):
        raise ValueError(f"W.codes {tuple(codes.shape)} and W.scales {tuple(scales.shape)} do not hold a {k} x {n} "
                         f"weight ({(groups, blocks, 16, 16)} and {(groups, blocks, 16)} do)")
    _need(codes, torch.uint8, "W.codes")
    _need_on(scales, scales.shape, torch.uint8, "W.scales", codes.device)
    return codes, scales, k, n, codes.device


def _rows(t, name: str) -> int:
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(t.shape)}")
    return t.shape[0]


def _rank(A) -> int:
    if A.dim() != 2:
        raise ValueError(f"A must be 2-D, got {tuple(A.shape)}")
    return A.shape[1]


def _out(t, shape, dtype, name: str, dev):
    if t is None:  # (with strides the call takes 1.2 us, without 1.6)
        strides = (shape[1], 1) if len(shape) == 2 else (shape[1] * 256, 256, 16, 1) if len(shape) == 4 else (shape[1] * 16, 16, 1)
        return torch.empty_strided(shape, strides, dtype=dtype, device=dev)
    _need_on(t, shape, dtype, name, dev)
    return t


def lora_mxfp4_quantize(W, *, codes=None, scales=None, stream=None) -> Mxfp4Weight:
    """W (k x n bf16) in MXFP4."""
    _need(W, _BF16, "W")
    k, n = _rows(W, "W"), W.shape[1]
    dev = W.device
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_mxfp4_quantize(W, codes=codes, scales=scales)
    groups, blocks = (n + 15) // 16, (k + 127) // 128 * 4
    codes = _out(codes, (groups, blocks, 16, 16), torch.uint8, "codes", dev)
    scales = _out(scales, (groups, blocks, 16), torch.uint8, "scales", dev)
    _check(load().lora_mxfp4_quantize(W.data_ptr(), k, n, codes.data_ptr(), scales.data_ptr(), _handle(dev)))
    return Mxfp4Weight(codes, scales, k, n)


def lora_mxfp4_dequantize(W: Mxfp4Weight, *, out=None, stream=None):
    """The k x n bf16 weight that W stands for (exact)."""
    codes, scales, k, n, dev = _need_weight(W)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_mxfp4_dequantize(W, out=out)
    out = _out(out, (k, n), _BF16, "out", dev)
    _check(load().lora_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), k, n, out.data_ptr(), _handle(dev)))
    return out


@_sizes
def lora_mxfp4_frozen_fwd_workspace_size(m, k, n) -> int:
    return load().lora_mxfp4_frozen_fwd_workspace_size(m, k, n)


@_sizes
def lora_mxfp4_frozen_bwd_workspace_size(m, k, n) -> int:
    return load().lora_mxfp4_frozen_bwd_workspace_size(m, k, n)


@_sizes
def lora_mxfp4_linear_fwd_workspace_size(m, k, n, r) -> int:
    return load().lora_mxfp4_linear_fwd_workspace_size(m, k, n, r)


@_sizes
def lora_mxfp4_linear_bwd_workspace_size(m, k, n, r) -> int:
    return load().lora_mxfp4_linear_bwd_workspace_size(m, k, n, r)


@_sizes
def multi_lora_mxfp4_fwd_workspace_size(m, k, n, r_max, num_adapters, num_segments) -> int:
    return load().multi_lora_mxfp4_fwd_workspace_size(m, k, n, r_max, num_adapters, num_segments)


@_sizes
def multi_lora_mxfp4_bwd_workspace_size(m, k, n, r_max, num_adapters, num_segments) -> int:
    return load().multi_lora_mxfp4_bwd_workspace_size(m, k, n, r_max, num_adapters, num_segments)


def lora_mxfp4_frozen_fwd(X, W: Mxfp4Weight, *, Y=None, workspace=None, stream=None):
    """Y = X W'."""
    codes, scales, k, n, dev = _need_weight(W)
    m = _rows(X, "X")
    _need_on(X, (m, k), _BF16, "X", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_mxfp4_frozen_fwd(X, W, Y=Y, workspace=workspace)
    lib = load()
    Y = _out(Y, (m, n), _BF16, "Y", dev)
    ws, nb, _held = _scratch(lora_mxfp4_frozen_fwd_workspace_size(m, k, n), dev, workspace)
    _check(lib.lora_mxfp4_frozen_fwd(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), m, k, n, Y.data_ptr(), ws, nb,
                                     _handle(dev)))
    return Y


def lora_mxfp4_frozen_bwd(dY, W: Mxfp4Weight, *, dX=None, workspace=None, stream=None):
    """dX = dY W'^T."""
    codes, scales, k, n, dev = _need_weight(W)
    m = _rows(dY, "dY")
    _need_on(dY, (m, n), _BF16, "dY", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_mxfp4_frozen_bwd(dY, W, dX=dX, workspace=workspace)
    lib = load()
    dX = _out(dX, (m, k), _BF16, "dX", dev)
    ws, nb, _held = _scratch(lora_mxfp4_frozen_bwd_workspace_size(m, k, n), dev, workspace)
    _check(lib.lora_mxfp4_frozen_bwd(dY.data_ptr(), codes.data_ptr(), scales.data_ptr(), m, k, n, dX.data_ptr(), ws, nb,
                                     _handle(dev)))
    return dX


def lora_mxfp4_linear_fwd(X, W: Mxfp4Weight, A, B, alpha: float, p: float, seed: int = 0, offset: int = 0, *,
                          Y=None, S=None, keep_bits=None, workspace=None, stream=None):
    """lora_linear_fwd over W'.  Returns (Y, S, keep_bits)."""
    codes, scales, k, n, dev = _need_weight(W)
    m, r = _rows(X, "X"), _rank(A)
    _need_on(X, (m, k), _BF16, "X", dev)
    _need_on(A, (k, r), _BF16, "A", dev)
    _need_on(B, (r, n), _BF16, "B", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_mxfp4_linear_fwd(X, W, A, B, alpha, p, seed, offset, Y=Y, S=S, keep_bits=keep_bits,
                                         workspace=workspace)
    lib = load()
    Y = _out(Y, (m, n), _BF16, "Y", dev)
    S = _out(S, (m, r), _F32, "S", dev)
    if keep_bits is not None or p != 0.0:
        keep_bits = _out(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    ws, nb, _held = _scratch(lora_mxfp4_linear_fwd_workspace_size(m, k, n, r), dev, workspace)
    _check(lib.lora_mxfp4_linear_fwd(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), A.data_ptr(), B.data_ptr(), m, k,
                                     n, r, alpha, p, seed, offset, Y.data_ptr(), S.data_ptr(),
                                     None if keep_bits is None else keep_bits.data_ptr(), ws, nb, _handle(dev)))
    return Y, S, keep_bits


def lora_mxfp4_linear_bwd(dY, X, W: Mxfp4Weight, A, B, S, keep_bits, alpha: float, p: float, *, dX=None, dA=None,
                          dB=None, workspace=None, stream=None, want_dX: bool = True):
    """lora_linear_bwd over W'.  Returns (dX, dA, dB); dX is None (and its
    product skipped) when want_dX is False."""
    codes, scales, k, n, dev = _need_weight(W)
    m, r = _rows(X, "X"), _rank(A)
    _need_on(X, (m, k), _BF16, "X", dev)
    _need_on(dY, (m, n), _BF16, "dY", dev)
    _need_on(A, (k, r), _BF16, "A", dev)
    _need_on(B, (r, n), _BF16, "B", dev)
    _need_on(S, (m, r), _F32, "S", dev)
    if keep_bits is not None:
        _need_on(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_mxfp4_linear_bwd(dY, X, W, A, B, S, keep_bits, alpha, p, dX=dX, dA=dA, dB=dB,
                                         workspace=workspace, want_dX=want_dX)
    lib = load()
    dX = _out(dX, (m, k), _BF16, "dX", dev) if want_dX else None
    dA = _out(dA, (k, r), _BF16, "dA", dev)
    dB = _out(dB, (r, n), _BF16, "dB", dev)
    ws, nb, _held = _scratch(lora_mxfp4_linear_bwd_workspace_size(m, k, n, r), dev, workspace)
    _check(lib.lora_mxfp4_linear_bwd(dY.data_ptr(), X.data_ptr(), codes.data_ptr(), scales.data_ptr(), A.data_ptr(),
                                     B.data_ptr(), S.data_ptr(), None if keep_bits is None else keep_bits.data_ptr(), m,
                                     k, n, r, alpha, p, None if dX is None else dX.data_ptr(), dA.data_ptr(),
                                     dB.data_ptr(), ws, nb, _handle(dev)))
    return dX, dA, dB


def _need_segments(seg_off, seg_adapter, adapters, num_adapters: int, k: int, n: int, r_max: int, dev) -> int:
    nseg = seg_adapter.numel()
    _need_on(seg_off, (nseg + 1,), torch.int64, "seg_off", dev)
    _need_on(seg_adapter, (nseg,), torch.int32, "seg_adapter", dev)
    _check_table(adapters, num_adapters, k, n, r_max)
    if adapters.device != dev:
        raise ValueError(f"adapters is on {adapters.device}, the weight on {dev}")
    return nseg


def multi_lora_mxfp4_linear_fwd(X, W: Mxfp4Weight, adapters: torch.Tensor, num_adapters: int, seg_off, seg_adapter,
                                r_max: int, seed: int = 0, offset: int = 0, *, Y=None, S=None, keep_bits=None,
                                workspace=None, stream=None):
    """multi_lora_linear_fwd over W'.  Returns (Y, S, keep_bits)."""
    codes, scales, k, n, dev = _need_weight(W)
    m = _rows(X, "X")
    _need_on(X, (m, k), _BF16, "X", dev)
    nseg = _need_segments(seg_off, seg_adapter, adapters, num_adapters, k, n, r_max, dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return multi_lora_mxfp4_linear_fwd(X, W, adapters, num_adapters, seg_off, seg_adapter, r_max, seed, offset,
                                               Y=Y, S=S, keep_bits=keep_bits, workspace=workspace)
    lib = load()
    Y = _out(Y, (m, n), _BF16, "Y", dev)
    S = _out(S, (m, r_max), _F32, "S", dev)
    keep_bits = _out(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    ws, nb, _held = _scratch(multi_lora_mxfp4_fwd_workspace_size(m, k, n, r_max, num_adapters, nseg), dev, workspace)
    _check(lib.multi_lora_mxfp4_linear_fwd(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), adapters.data_ptr(),
                                           num_adapters, seg_off.data_ptr(), seg_adapter.data_ptr(), nseg, m, k, n,
                                           r_max, seed, offset, Y.data_ptr(), S.data_ptr(), keep_bits.data_ptr(), ws, nb,
                                           _handle(dev)))
    return Y, S, keep_bits


def multi_lora_mxfp4_linear_bwd(dY, X, W: Mxfp4Weight, adapters: torch.Tensor, num_adapters: int, seg_off,
                                seg_adapter, S, keep_bits, r_max: int, *, dX=None, workspace=None, stream=None,
                                want_dX: bool = True) -> Optional[torch.Tensor]:
    """multi_lora_linear_bwd over W': writes the table's dA and dB, returns dX
    (None, its product skipped, when want_dX is False)."""
    codes, scales, k, n, dev = _need_weight(W)
    m = _rows(X, "X")
    _need_on(X, (m, k), _BF16, "X", dev)
    nseg = _need_segments(seg_off, seg_adapter, adapters, num_adapters, k, n, r_max, dev)
    _need_on(dY, (m, n), _BF16, "dY", dev)
    _need_on(S, (m, r_max), _F32, "S", dev)
    _need_on(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return multi_lora_mxfp4_linear_bwd(dY, X, W, adapters, num_adapters, seg_off, seg_adapter, S, keep_bits,
                                               r_max, dX=dX, workspace=workspace, want_dX=want_dX)
    lib = load()
    dX = _out(dX, (m, k), _BF16, "dX", dev) if want_dX else None
    ws, nb, _held = _scratch(multi_lora_mxfp4_bwd_workspace_size(m, k, n, r_max, num_adapters, nseg), dev, workspace)
    _check(lib.multi_lora_mxfp4_linear_bwd(dY.data_ptr(), X.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                           adapters.data_ptr(), num_adapters, seg_off.data_ptr(), seg_adapter.data_ptr(),
                                           nseg, S.data_ptr(), keep_bits.data_ptr(), m, k, n, r_max,
                                           None if dX is None else dX.data_ptr(), ws, nb, _handle(dev)))
    return dX
