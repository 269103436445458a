"""Frozen weights of 4-bit integers in groups of rows and the layers over them.

Every function has the name of a C-ABI entry point in include/lora_fused.h and
only marshals arguments, as the rest of the binding does.  `lora_linear`,
`multi_lora_linear` and `LoraLinear` take an Int4Weight wherever they take W.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch

from ._lib import (_check, _check_table, _elsewhere, _handle, _need, _need_on, _on_device, _scratch, load)

_BF16, _F32 = torch.bfloat16, torch.float32
_SCALE_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_sizes = functools.lru_cache(maxsize=1024)  # sizes follow from what is asked for alone


class Int4Weight(NamedTuple):
    """A frozen k x n weight s (q - z) of 4-bit integers q with one scale s and
    zero z for `group` rows of a column.  `codes` (ceil(n/16), ceil(k/128), 4,
    16, 16) uint8 and `scales` (ceil(n/16), G, 16) int32 are device tensors as
    include/lora_fused.h describes them; lora_int4_quantize makes them from a
    bf16 weight, lora_int4_pack from a checkpoint's integers, scales and zeros."""
    codes: torch.Tensor
    scales: torch.Tensor
    k: int
    n: int
    group: int

    @property
    def shape(self):
        return (self.k, self.n)

    @property
    def device(self):
        return self.codes.device


@_sizes
def _shapes(k: int, n: int, group: int):
    """Shapes of a weight's codes and scales."""
    wide, deep = (n + 15) // 16, (k + 127) // 128
    if group not in (32, 64) and (group <= 0 or group % 128):
        raise ValueError(f"group = {group} must be 32, 64 or a multiple of 128")
    return (wide, deep, 4, 16, 16), (wide, deep * 128 // group if group < 128 else -(-k // group), 16)


def _need_weight(W: Int4Weight):
    if not isinstance(W, Int4Weight):
        raise TypeError(f"W must be an Int4Weight, got {type(W).__name__}")
    codes, scales, k, n, group = W
    c, s = _shapes(k, n, group)
    if (codes.shape == c and scales.shape == s and codes.is_cuda and codes.dtype is torch.uint8
            and scales.dtype is torch.int32 and codes.is_contiguous() and scales.is_contiguous()
            and scales.get_device() == codes.get_device()):
        return codes, scales, k, n, group, codes.device
    if codes.shape != c or scales.shape != s:
        raise ValueError(f"W.codes {tuple(codes.shape)} and W.scales {tuple(scales.shape)} do not hold a {k} x {n} "
                         f"weight in groups of {group} ({c} and {s} do)")
    _need(codes, torch.uint8, "W.codes")
    _need_on(scales, s, torch.int32, "W.scales", codes.device)
    return codes, scales, k, n, group, codes.device


def _matrix(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(t.shape)}")
    return t.shape


def _out(t, shape, dtype, name: str, dev):
    if t is None:
        if len(shape) < 4:  # (with strides the call takes 1.0 us, without 1.4)
            strides = (shape[1], 1) if len(shape) == 2 else (shape[1] * shape[2], shape[2], 1)
            return torch.empty_strided(shape, strides, dtype=dtype, device=dev)
        return torch.empty(shape, dtype=dtype, device=dev)
    _need_on(t, shape, dtype, name, dev)
    return t


def lora_int4_quantize(W, group: int = 128, *, symmetric: bool = False, codes=None, scales=None,
                       stream=None) -> Int4Weight:
    """W (k x n bf16) as 4-bit integers: to the nearest, with a scale and a zero
    (symmetric: the zero is 8) for `group` rows of a column."""
    _need(W, _BF16, "W")
    k, n = _matrix(W, "W")
    dev = W.device
    c, s = _shapes(k, n, group)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_int4_quantize(W, group, symmetric=symmetric, codes=codes, scales=scales)
    codes, scales = _out(codes, c, torch.uint8, "codes", dev), _out(scales, s, torch.int32, "scales", dev)
    _check(load().lora_int4_quantize(W.data_ptr(), k, n, group, bool(symmetric), codes.data_ptr(), scales.data_ptr(),
                                     _handle(dev)))
    return Int4Weight(codes, scales, k, n, group)


def lora_int4_pack(Q, group_scales, zeros=None, *, group: int, codes=None, scales=None, stream=None) -> Int4Weight:
    """A checkpoint's weight: Q (k x n uint8, a code of 0 .. 15 each),
    group_scales (ceil(k/group) x n, fp32, bf16 or fp16) and zeros (the same
    shape, uint8; None: every zero is 8)."""
    _need(Q, torch.uint8, "Q")
    k, n = _matrix(Q, "Q")
    dev = Q.device
    c, s = _shapes(k, n, group)
    given = torch.Size((-(-k // group), n))
    if group_scales.dtype not in _SCALE_TYPES:
        raise TypeError(f"group_scales must be float32, bfloat16 or float16, got {group_scales.dtype}")
    _need_on(group_scales, given, group_scales.dtype, "group_scales", dev)
    if zeros is not None:
        _need_on(zeros, given, torch.uint8, "zeros", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_int4_pack(Q, group_scales, zeros, group=group, codes=codes, scales=scales)
    codes, scales = _out(codes, c, torch.uint8, "codes", dev), _out(scales, s, torch.int32, "scales", dev)
    _check(load().lora_int4_pack(Q.data_ptr(), group_scales.data_ptr(), _SCALE_TYPES[group_scales.dtype],
                                 None if zeros is None else zeros.data_ptr(), k, n, group, codes.data_ptr(),
                                 scales.data_ptr(), _handle(dev)))
    return Int4Weight(codes, scales, k, n, group)


def lora_int4_dequantize(W: Int4Weight, *, out=None, stream=None):
    """The k x n weight that W stands for, each value rounded to bf16."""
    codes, scales, k, n, group, dev = _need_weight(W)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_int4_dequantize(W, out=out)
    out = _out(out, (k, n), _BF16, "out", dev)
    _check(load().lora_int4_dequantize(codes.data_ptr(), scales.data_ptr(), k, n, group, out.data_ptr(), _handle(dev)))
    return out


@_sizes
def lora_int4_frozen_fwd_workspace_size(m, k, n, group) -> int:
    return load().lora_int4_frozen_fwd_workspace_size(m, k, n, group)


@_sizes
def lora_int4_frozen_bwd_workspace_size(m, k, n, group) -> int:
    return load().lora_int4_frozen_bwd_workspace_size(m, k, n, group)


@_sizes
def lora_int4_linear_fwd_workspace_size(m, k, n, group, r) -> int:
    return load().lora_int4_linear_fwd_workspace_size(m, k, n, group, r)


@_sizes
def lora_int4_linear_bwd_workspace_size(m, k, n, group, r) -> int:
    return load().lora_int4_linear_bwd_workspace_size(m, k, n, group, r)


@_sizes
def multi_lora_int4_fwd_workspace_size(m, k, n, group, r_max, num_adapters, num_segments) -> int:
    return load().multi_lora_int4_fwd_workspace_size(m, k, n, group, r_max, num_adapters, num_segments)


@_sizes
def multi_lora_int4_bwd_workspace_size(m, k, n, group, r_max, num_adapters, num_segments) -> int:
    return load().multi_lora_int4_bwd_workspace_size(m, k, n, group, r_max, num_adapters, num_segments)


def lora_int4_frozen_fwd(X, W: Int4Weight, *, Y=None, workspace=None, stream=None):
    """Y = X W'."""
    codes, scales, k, n, group, dev = _need_weight(W)
    m = _matrix(X, "X")[0]
    _need_on(X, (m, k), _BF16, "X", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_int4_frozen_fwd(X, W, Y=Y, workspace=workspace)
    Y = _out(Y, (m, n), _BF16, "Y", dev)
    ws, nb, _held = _scratch(lora_int4_frozen_fwd_workspace_size(m, k, n, group), dev, workspace)
    _check(load().lora_int4_frozen_fwd(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), group, m, k, n, Y.data_ptr(),
                                       ws, nb, _handle(dev)))
    return Y


def lora_int4_frozen_bwd(dY, W: Int4Weight, *, dX=None, workspace=None, stream=None):
    """dX = dY W'^T."""
    codes, scales, k, n, group, dev = _need_weight(W)
    m = _matrix(dY, "dY")[0]
    _need_on(dY, (m, n), _BF16, "dY", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_int4_frozen_bwd(dY, W, dX=dX, workspace=workspace)
    dX = _out(dX, (m, k), _BF16, "dX", dev)
    ws, nb, _held = _scratch(lora_int4_frozen_bwd_workspace_size(m, k, n, group), dev, workspace)
    _check(load().lora_int4_frozen_bwd(dY.data_ptr(), codes.data_ptr(), scales.data_ptr(), group, m, k, n,
                                       dX.data_ptr(), ws, nb, _handle(dev)))
    return dX


def lora_int4_linear_fwd(X, W: Int4Weight, A, B, alpha: float, p: float, seed: int = 0, offset: int = 0, *,
                         Y=None, S=None, keep_bits=None, workspace=None, stream=None):
    """lora_linear_fwd over W'.  Returns (Y, S, keep_bits)."""
    codes, scales, k, n, group, dev = _need_weight(W)
    m, r = _matrix(X, "X")[0], _matrix(A, "A")[1]
    _need_on(X, (m, k), _BF16, "X", dev)
    _need_on(A, (k, r), _BF16, "A", dev)
    _need_on(B, (r, n), _BF16, "B", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_int4_linear_fwd(X, W, A, B, alpha, p, seed, offset, Y=Y, S=S, keep_bits=keep_bits,
                                        workspace=workspace)
    Y = _out(Y, (m, n), _BF16, "Y", dev)
    S = _out(S, (m, r), _F32, "S", dev)
    if keep_bits is not None or p != 0.0:
        keep_bits = _out(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    ws, nb, _held = _scratch(lora_int4_linear_fwd_workspace_size(m, k, n, group, r), dev, workspace)
    _check(load().lora_int4_linear_fwd(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), group, A.data_ptr(),
                                       B.data_ptr(), m, k, n, r, alpha, p, seed, offset, Y.data_ptr(), S.data_ptr(),
                                       None if keep_bits is None else keep_bits.data_ptr(), ws, nb, _handle(dev)))
    return Y, S, keep_bits


def lora_int4_linear_bwd(dY, X, W: Int4Weight, A, B, S, keep_bits, alpha: float, p: float, *, dX=None, dA=None,
                         dB=None, workspace=None, stream=None, want_dX: bool = True):
    """lora_linear_bwd over W'.  Returns (dX, dA, dB); dX is None (and its
    product skipped) when want_dX is False."""
    codes, scales, k, n, group, dev = _need_weight(W)
    m, r = _matrix(X, "X")[0], _matrix(A, "A")[1]
    _need_on(X, (m, k), _BF16, "X", dev)
    _need_on(dY, (m, n), _BF16, "dY", dev)
    _need_on(A, (k, r), _BF16, "A", dev)
    _need_on(B, (r, n), _BF16, "B", dev)
    _need_on(S, (m, r), _F32, "S", dev)
    if keep_bits is not None:
        _need_on(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return lora_int4_linear_bwd(dY, X, W, A, B, S, keep_bits, alpha, p, dX=dX, dA=dA, dB=dB,
                                        workspace=workspace, want_dX=want_dX)
    dX = _out(dX, (m, k), _BF16, "dX", dev) if want_dX else None
    dA = _out(dA, (k, r), _BF16, "dA", dev)
    dB = _out(dB, (r, n), _BF16, "dB", dev)
    ws, nb, _held = _scratch(lora_int4_linear_bwd_workspace_size(m, k, n, group, r), dev, workspace)
    _check(load().lora_int4_linear_bwd(dY.data_ptr(), X.data_ptr(), codes.data_ptr(), scales.data_ptr(), group,
                                       A.data_ptr(), B.data_ptr(), S.data_ptr(),
                                       None if keep_bits is None else keep_bits.data_ptr(), m, k, n, r, alpha, p,
                                       None if dX is None else dX.data_ptr(), dA.data_ptr(), dB.data_ptr(), ws, nb,
                                       _handle(dev)))
    return dX, dA, dB


def _need_segments(seg_off, seg_adapter, adapters, num_adapters: int, k: int, n: int, r_max: int, dev) -> int:
    nseg = seg_adapter.numel()
    _need_on(seg_off, (nseg + 1,), torch.int64, "seg_off", dev)
    _need_on(seg_adapter, (nseg,), torch.int32, "seg_adapter", dev)
    _check_table(adapters, num_adapters, k, n, r_max)
    if adapters.device != dev:
        raise ValueError(f"adapters is on {adapters.device}, the weight on {dev}")
    return nseg


def multi_lora_int4_linear_fwd(X, W: Int4Weight, adapters: torch.Tensor, num_adapters: int, seg_off, seg_adapter,
                               r_max: int, seed: int = 0, offset: int = 0, *, Y=None, S=None, keep_bits=None,
                               workspace=None, stream=None):
    """multi_lora_linear_fwd over W'.  Returns (Y, S, keep_bits)."""
    codes, scales, k, n, group, dev = _need_weight(W)
    m = _matrix(X, "X")[0]
    _need_on(X, (m, k), _BF16, "X", dev)
    nseg = _need_segments(seg_off, seg_adapter, adapters, num_adapters, k, n, r_max, dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return multi_lora_int4_linear_fwd(X, W, adapters, num_adapters, seg_off, seg_adapter, r_max, seed, offset,
                                              Y=Y, S=S, keep_bits=keep_bits, workspace=workspace)
    Y = _out(Y, (m, n), _BF16, "Y", dev)
    S = _out(S, (m, r_max), _F32, "S", dev)
    keep_bits = _out(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    ws, nb, _held = _scratch(multi_lora_int4_fwd_workspace_size(m, k, n, group, r_max, num_adapters, nseg), dev,
                             workspace)
    _check(load().multi_lora_int4_linear_fwd(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), group,
                                             adapters.data_ptr(), num_adapters, seg_off.data_ptr(),
                                             seg_adapter.data_ptr(), nseg, m, k, n, r_max, seed, offset, Y.data_ptr(),
                                             S.data_ptr(), keep_bits.data_ptr(), ws, nb, _handle(dev)))
    return Y, S, keep_bits


def multi_lora_int4_linear_bwd(dY, X, W: Int4Weight, adapters: torch.Tensor, num_adapters: int, seg_off, seg_adapter,
                               S, keep_bits, r_max: int, *, dX=None, workspace=None, stream=None,
                               want_dX: bool = True) -> Optional[torch.Tensor]:
    """multi_lora_linear_bwd over W': writes the table's dA and dB, returns dX
    (None, its product skipped, when want_dX is False)."""
    codes, scales, k, n, group, dev = _need_weight(W)
    m = _matrix(X, "X")[0]
    _need_on(X, (m, k), _BF16, "X", dev)
    nseg = _need_segments(seg_off, seg_adapter, adapters, num_adapters, k, n, r_max, dev)
    _need_on(dY, (m, n), _BF16, "dY", dev)
    _need_on(S, (m, r_max), _F32, "S", dev)
    _need_on(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    if _elsewhere(dev, stream):
        with _on_device(dev, stream):
            return multi_lora_int4_linear_bwd(dY, X, W, adapters, num_adapters, seg_off, seg_adapter, S, keep_bits,
                                              r_max, dX=dX, workspace=workspace, want_dX=want_dX)
    dX = _out(dX, (m, k), _BF16, "dX", dev) if want_dX else None
    ws, nb, _held = _scratch(multi_lora_int4_bwd_workspace_size(m, k, n, group, r_max, num_adapters, nseg), dev,
                             workspace)
    _check(load().multi_lora_int4_linear_bwd(dY.data_ptr(), X.data_ptr(), codes.data_ptr(), scales.data_ptr(), group,
                                             adapters.data_ptr(), num_adapters, seg_off.data_ptr(),
                                             seg_adapter.data_ptr(), nseg, S.data_ptr(), keep_bits.data_ptr(), m, k, n,
                                             r_max, None if dX is None else dX.data_ptr(), ws, nb, _handle(dev)))
    return dX
