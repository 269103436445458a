"""Frozen weights held in 4 bits (MXFP4) and the layers over them.

Every function has the name of a C-ABI entry point in include/lora_fused.h and
only marshals arguments, as the rest of the binding does.  `lora_linear`,
`multi_lora_linear` and `LoraLinear` take an Mxfp4Weight wherever they take W.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from ._lib import _check, _check_table, _need, _on_device, _ptr, _scratch, load


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


def _storage(k: int, n: int):
    return (n + 15) // 16, (k + 127) // 128 * 4, 16


def _need_weight(W: Mxfp4Weight):
    if not isinstance(W, Mxfp4Weight):
        raise TypeError(f"W must be an Mxfp4Weight, got {type(W).__name__}")
    codes, scales, k, n = W
    _need(codes, torch.uint8, "W.codes")
    _need(scales, torch.uint8, "W.scales")
    at = _storage(k, n)
    if codes.shape != at + (16,) or scales.shape != at:
        raise ValueError(f"W.codes {tuple(codes.shape)} and W.scales {tuple(scales.shape)} do not hold a "
                         f"{k} x {n} weight ({at + (16,)} and {at} do)")
    return codes, scales, k, n


def _need_rows(t, width: int, name: str, dev, dtype=torch.bfloat16) -> int:
    """Rows of a contiguous (rows, width) tensor on `dev`."""
    _need(t, dtype, name)
    if t.dim() != 2 or t.shape[1] != width:
        raise ValueError(f"{name} must be (rows, {width}), got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the weight on {dev}")
    return t.shape[0]


def _need_shape(t, shape, dtype, name: str, dev) -> None:
    _need(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the weight on {dev}")


def _out(t, shape, dtype, name: str, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need_shape(t, shape, dtype, name, dev)
    return t


def _need_keep(keep, m: int, k: int, dev) -> None:
    if keep is not None:
        _need_shape(keep, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)


def lora_mxfp4_quantize(W, *, codes=None, scales=None, stream=None) -> Mxfp4Weight:
    """W (k x n bf16) in MXFP4."""
    _need(W, torch.bfloat16, "W")
    if W.dim() != 2:
        raise ValueError(f"W must be 2-D, got {tuple(W.shape)}")
    k, n = W.shape
    dev = W.device
    with _on_device(dev, stream) as st:
        codes = _out(codes, _storage(k, n) + (16,), torch.uint8, "codes", dev)
        scales = _out(scales, _storage(k, n), torch.uint8, "scales", dev)
        _check(load().lora_mxfp4_quantize(_ptr(W), k, n, _ptr(codes), _ptr(scales), st))
    return Mxfp4Weight(codes, scales, k, n)


def lora_mxfp4_dequantize(W: Mxfp4Weight, *, out=None, stream=None):
    """The k x n bf16 weight that W stands for (exact)."""
    codes, scales, k, n = _need_weight(W)
    dev = codes.device
    with _on_device(dev, stream) as st:
        out = _out(out, (k, n), torch.bfloat16, "out", dev)
        _check(load().lora_mxfp4_dequantize(_ptr(codes), _ptr(scales), k, n, _ptr(out), st))
    return out


def lora_mxfp4_frozen_fwd_workspace_size(m, k, n) -> int:
    return int(load().lora_mxfp4_frozen_fwd_workspace_size(m, k, n))


def lora_mxfp4_frozen_bwd_workspace_size(m, k, n) -> int:
    return int(load().lora_mxfp4_frozen_bwd_workspace_size(m, k, n))


def lora_mxfp4_linear_fwd_workspace_size(m, k, n, r) -> int:
    return int(load().lora_mxfp4_linear_fwd_workspace_size(m, k, n, r))


def lora_mxfp4_linear_bwd_workspace_size(m, k, n, r) -> int:
    return int(load().lora_mxfp4_linear_bwd_workspace_size(m, k, n, r))


def multi_lora_mxfp4_fwd_workspace_size(m, k, n, r_max, num_adapters, num_segments) -> int:
    return int(load().multi_lora_mxfp4_fwd_workspace_size(m, k, n, r_max, num_adapters, num_segments))


def multi_lora_mxfp4_bwd_workspace_size(m, k, n, r_max, num_adapters, num_segments) -> int:
    return int(load().multi_lora_mxfp4_bwd_workspace_size(m, k, n, r_max, num_adapters, num_segments))


def lora_mxfp4_frozen_fwd(X, W: Mxfp4Weight, *, Y=None, workspace=None, stream=None):
    """Y = X W'."""
    codes, scales, k, n = _need_weight(W)
    dev = codes.device
    m = _need_rows(X, k, "X", dev)
    with _on_device(dev, stream) as st:
        Y = _out(Y, (m, n), torch.bfloat16, "Y", dev)
        ws, nb = _scratch(lora_mxfp4_frozen_fwd_workspace_size(m, k, n), dev, workspace)
        _check(load().lora_mxfp4_frozen_fwd(_ptr(X), _ptr(codes), _ptr(scales), m, k, n, _ptr(Y), ws, nb, st))
    return Y


def lora_mxfp4_frozen_bwd(dY, W: Mxfp4Weight, *, dX=None, workspace=None, stream=None):
    """dX = dY W'^T."""
    codes, scales, k, n = _need_weight(W)
    dev = codes.device
    m = _need_rows(dY, n, "dY", dev)
    with _on_device(dev, stream) as st:
        dX = _out(dX, (m, k), torch.bfloat16, "dX", dev)
        ws, nb = _scratch(lora_mxfp4_frozen_bwd_workspace_size(m, k, n), dev, workspace)
        _check(load().lora_mxfp4_frozen_bwd(_ptr(dY), _ptr(codes), _ptr(scales), m, k, n, _ptr(dX), ws, nb, st))
    return dX


def lora_mxfp4_linear_fwd(X, W: Mxfp4Weight, A, B, alpha: float, p: float, seed: int = 0, offset: int = 0, *,
                          Y=None, S=None, keep_bits=None, workspace=None, stream=None):
    """lora_linear_fwd over W'.  Returns (Y, S, keep_bits)."""
    codes, scales, k, n = _need_weight(W)
    dev = codes.device
    m = _need_rows(X, k, "X", dev)
    r = A.shape[1] if A.dim() == 2 else 0
    _need_shape(A, (k, r), torch.bfloat16, "A", dev)
    _need_shape(B, (r, n), torch.bfloat16, "B", dev)
    _need_keep(keep_bits, m, k, dev)
    with _on_device(dev, stream) as st:
        Y = _out(Y, (m, n), torch.bfloat16, "Y", dev)
        S = _out(S, (m, r), torch.float32, "S", dev)
        if keep_bits is None and p != 0.0:
            keep_bits = torch.empty((m, (k + 31) // 32), dtype=torch.int32, device=dev)
        ws, nb = _scratch(lora_mxfp4_linear_fwd_workspace_size(m, k, n, r), dev, workspace)
        _check(load().lora_mxfp4_linear_fwd(_ptr(X), _ptr(codes), _ptr(scales), _ptr(A), _ptr(B), m, k, n, r, alpha,
                                            p, seed, offset, _ptr(Y), _ptr(S), _ptr(keep_bits), ws, nb, st))
    return Y, S, keep_bits


def lora_mxfp4_linear_bwd(dY, X, W: Mxfp4Weight, A, B, S, keep_bits, alpha: float, p: float, *, dX=None, dA=None,
                          dB=None, workspace=None, stream=None, want_dX: bool = True):
    """lora_linear_bwd over W'.  Returns (dX, dA, dB); dX is None (and its
    product skipped) when want_dX is False."""
    codes, scales, k, n = _need_weight(W)
    dev = codes.device
    m = _need_rows(X, k, "X", dev)
    r = A.shape[1] if A.dim() == 2 else 0
    _need_shape(dY, (m, n), torch.bfloat16, "dY", dev)
    _need_shape(A, (k, r), torch.bfloat16, "A", dev)
    _need_shape(B, (r, n), torch.bfloat16, "B", dev)
    _need_shape(S, (m, r), torch.float32, "S", dev)
    _need_keep(keep_bits, m, k, dev)
    with _on_device(dev, stream) as st:
        dX = _out(dX, (m, k), torch.bfloat16, "dX", dev) if want_dX else None
        dA = _out(dA, (k, r), torch.bfloat16, "dA", dev)
        dB = _out(dB, (r, n), torch.bfloat16, "dB", dev)
        ws, nb = _scratch(lora_mxfp4_linear_bwd_workspace_size(m, k, n, r), dev, workspace)
        _check(load().lora_mxfp4_linear_bwd(_ptr(dY), _ptr(X), _ptr(codes), _ptr(scales), _ptr(A), _ptr(B), _ptr(S),
                                            _ptr(keep_bits), m, k, n, r, alpha, p, _ptr(dX), _ptr(dA), _ptr(dB), ws,
                                            nb, st))
    return dX, dA, dB


def _need_segments(seg_off, seg_adapter, adapters, num_adapters: int, k: int, n: int, r_max: int, dev) -> int:
    _need(seg_off, torch.int64, "seg_off")
    _need(seg_adapter, torch.int32, "seg_adapter")
    _check_table(adapters, num_adapters, k, n, r_max)
    nseg = seg_adapter.numel()
    if seg_off.numel() != nseg + 1:
        raise ValueError(f"seg_off must have {nseg + 1} entries for {nseg} segments, got {seg_off.numel()}")
    for t, nm in ((seg_off, "seg_off"), (seg_adapter, "seg_adapter"), (adapters, "adapters")):
        if t.device != dev:
            raise ValueError(f"{nm} is on {t.device}, the weight on {dev}")
    return nseg


def multi_lora_mxfp4_linear_fwd(X, W: Mxfp4Weight, adapters: torch.Tensor, num_adapters: int, seg_off, seg_adapter,
                                r_max: int, seed: int = 0, offset: int = 0, *, Y=None, S=None, keep_bits=None,
                                workspace=None, stream=None):
    """multi_lora_linear_fwd over W'.  Returns (Y, S, keep_bits)."""
    codes, scales, k, n = _need_weight(W)
    dev = codes.device
    m = _need_rows(X, k, "X", dev)
    nseg = _need_segments(seg_off, seg_adapter, adapters, num_adapters, k, n, r_max, dev)
    with _on_device(dev, stream) as st:
        Y = _out(Y, (m, n), torch.bfloat16, "Y", dev)
        S = _out(S, (m, r_max), torch.float32, "S", dev)
        keep_bits = _out(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
        ws, nb = _scratch(multi_lora_mxfp4_fwd_workspace_size(m, k, n, r_max, num_adapters, nseg), dev, workspace)
        _check(load().multi_lora_mxfp4_linear_fwd(_ptr(X), _ptr(codes), _ptr(scales), _ptr(adapters), num_adapters,
                                                  _ptr(seg_off), _ptr(seg_adapter), nseg, m, k, n, r_max, seed,
                                                  offset, _ptr(Y), _ptr(S), _ptr(keep_bits), ws, nb, st))
    return Y, S, keep_bits


def multi_lora_mxfp4_linear_bwd(dY, X, W: Mxfp4Weight, adapters: torch.Tensor, num_adapters: int, seg_off,
                                seg_adapter, S, keep_bits, r_max: int, *, dX=None, workspace=None, stream=None,
                                want_dX: bool = True) -> Optional[torch.Tensor]:
    """multi_lora_linear_bwd over W': writes the table's dA and dB, returns dX
    (None, its product skipped, when want_dX is False)."""
    codes, scales, k, n = _need_weight(W)
    dev = codes.device
    m = _need_rows(X, k, "X", dev)
    nseg = _need_segments(seg_off, seg_adapter, adapters, num_adapters, k, n, r_max, dev)
    _need_shape(dY, (m, n), torch.bfloat16, "dY", dev)
    _need_shape(S, (m, r_max), torch.float32, "S", dev)
    _need_shape(keep_bits, (m, (k + 31) // 32), torch.int32, "keep_bits", dev)
    with _on_device(dev, stream) as st:
        dX = _out(dX, (m, k), torch.bfloat16, "dX", dev) if want_dX else None
        ws, nb = _scratch(multi_lora_mxfp4_bwd_workspace_size(m, k, n, r_max, num_adapters, nseg), dev, workspace)
        _check(load().multi_lora_mxfp4_linear_bwd(_ptr(dY), _ptr(X), _ptr(codes), _ptr(scales), _ptr(adapters),
                                                  num_adapters, _ptr(seg_off), _ptr(seg_adapter), nseg, _ptr(S),
                                                  _ptr(keep_bits), m, k, n, r_max, _ptr(dX), ws, nb, st))
    return dX
