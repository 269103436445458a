"""PyTorch autograd glue over the C ABI: the LoRA linear layer as a
torch.autograd.Function and a module holding a frozen weight and one adapter.

The forward saves what the library's backward consumes (X, S and the mask
bits; W, A and B by reference), so the layer drops in where a PEFT-style LoRA
layer sits (juhe.plus blog on LoRAFusion, section 6: the fused kernels plug
into existing LoRA stacks as replacements).  Every step runs in the library;
this file only reshapes tensors and keeps the dropout counter.
"""
from __future__ import annotations

from collections import OrderedDict

import torch

from . import _lib, int4, mxfp4, mxint8
from .int4 import Int4Weight
from .mxfp4 import Mxfp4Weight
from .mxint8 import Mxint8Input


def _weight_tensors(W):
    """The tensors of a frozen weight (one bf16 tensor, or a packed weight's two)."""
    return (W.codes, W.scales) if isinstance(W, (Mxfp4Weight, Int4Weight)) else (W,)


def _weight_again(tensors, k: int, n: int, group: int = 0):
    """The weight of these tensors (group: an Int4Weight's, else 0)."""
    if len(tensors) == 1:
        return tensors[0]
    return Int4Weight(*tensors, k, n, group) if group else Mxfp4Weight(*tensors, k, n)


def _of(W, name: str):
    """The binding's call `name` for a weight of W's form."""
    if isinstance(W, Mxfp4Weight):
        return getattr(mxfp4, name.replace("lora_", "lora_mxfp4_", 1))
    if isinstance(W, Int4Weight):
        return getattr(int4, name.replace("lora_", "lora_int4_", 1))
    return getattr(_lib, name)


def _input_tensors(X, X8):
    """What the backward keeps of an input: itself, or its 8-bit copy's two tensors."""
    if X8 is None:
        return (X,)
    if not isinstance(X8, Mxint8Input):
        raise TypeError(f"X8 must be an Mxint8Input, got {type(X8).__name__}")
    if X8.shape != tuple(X.shape) or X8.device != X.device:
        raise ValueError(f"X8 holds {tuple(X8.shape)} on {X8.device}, X is {tuple(X.shape)} on {X.device}")
    return X8.codes, X8.scales


class LoraLinearFunction(torch.autograd.Function):
    """Y = X W + alpha * (dropout(X) A) B for X (..., k) bf16; W k x n, a bf16
    tensor, an Mxfp4Weight or an Int4Weight, is frozen (no gradient); A k x r and
    B r x n receive gradients.  With X8, X's rows saved in 8 bits, the backward
    keeps those instead of X."""

    @staticmethod
    def forward(ctx, X, W, A, B, alpha: float, p: float, seed: int, offset: int, X8=None):
        lead = X.shape[:-1]
        X2 = X.reshape(-1, X.shape[-1]).contiguous()
        kept = _input_tensors(X2, X8)
        Y, S, keep = _of(W, "lora_linear_fwd")(X2, W, A, B, alpha, p, seed, offset)
        ctx.save_for_backward(A, B, S, keep if keep is not None else torch.empty(0, device=X.device), *kept,
                              *_weight_tensors(W))
        ctx.alpha, ctx.p, ctx.lead, ctx.has_keep = alpha, p, lead, keep is not None
        ctx.kept, ctx.k, ctx.group = len(kept), X2.shape[1], getattr(W, "group", 0)
        return Y.reshape(*lead, W.shape[1])

    @staticmethod
    def backward(ctx, dY):
        A, B, S, keep, *rest = ctx.saved_tensors
        W = _weight_again(rest[ctx.kept:], ctx.k, B.shape[1], ctx.group)
        dY2 = dY.reshape(-1, dY.shape[-1]).contiguous()
        want_dX = ctx.needs_input_grad[0]
        if ctx.kept == 1:
            bwd, X = _of(W, "lora_linear_bwd"), rest[0]
        else:
            bwd, X = mxint8.lora_mxint8_linear_bwd, Mxint8Input(*rest[:2], ctx.k)
        dX, dA, dB = bwd(dY2, X, W, A, B, S, keep if ctx.has_keep else None, ctx.alpha, ctx.p, want_dX=want_dX)
        dX = dX.reshape(*ctx.lead, ctx.k) if want_dX else None
        return dX, None, dA, dB, None, None, None, None, None


def lora_linear(X, W, A, B, alpha: float, p: float = 0.0, seed: int = 0, offset: int = 0, X8=None):
    """The layer as an autograd function.  X8 (lora_mxint8_quantize of X's rows) is
    what the backward keeps in X's place; layers that share an input share it."""
    return LoraLinearFunction.apply(X, W, A, B, alpha, p, seed, offset, X8)


class _AdapterSet:
    """The device adapter table of one set of adapter tensors, built once and
    reused by every call with the same tensors, scales and dropout ratios.

    The backward writes all gradients of the set into one flat bf16 buffer per
    call; the table's dA / dB pointer slots are set to that buffer's pieces
    by one device-side add (constant piece offsets plus the buffer's base
    address, a kernel argument), so no call after the first copies from host
    memory or waits for the device, and the calls can be captured in a graph.
    Calls that share a set must run in stream order (one stream)."""

    def __init__(self, As, Bs, alphas, ps):
        self.table = _lib.adapter_table(As, Bs, alphas, ps)
        self.k, self.n, ranks = self.table._lora_meta
        self.num = len(As)
        self.r_max = max(ranks)
        self.shapes = [(tuple(a.shape), tuple(b.shape)) for a, b in zip(As, Bs)]
        offs, pos = [], 0
        for sa, sb in self.shapes:
            na, nb = sa[0] * sa[1], sb[0] * sb[1]
            offs.append((pos, pos + (na + 7) // 8 * 8))  # pieces start on 16-byte boundaries
            pos += (na + 7) // 8 * 8 + (nb + 7) // 8 * 8
        self.total = pos
        self.elem_off = offs
        self.byte_off = torch.tensor([[2 * a, 2 * b] for a, b in offs], dtype=torch.int64,
                                     device=self.table.device)

    def gradient_buffers(self):
        flat = torch.empty(max(self.total, 1), dtype=torch.bfloat16, device=self.table.device)
        slots = self.table.view(torch.int64).view(self.num, 6)[:, 2:4]  # dA, dB of each record
        torch.add(self.byte_off, flat.data_ptr(), out=slots)
        dAs, dBs = [], []
        for (oa, ob), (sa, sb) in zip(self.elem_off, self.shapes):
            dAs.append(flat[oa:oa + sa[0] * sa[1]].view(sa))
            dBs.append(flat[ob:ob + sb[0] * sb[1]].view(sb))
        return dAs, dBs


_SETS: "OrderedDict[tuple, _AdapterSet]" = OrderedDict()
_SETS_MAX = 256


def _adapter_set(As, Bs, alphas, ps) -> _AdapterSet:
    # layout is part of the key: a tensor that would fail the checks never hits the cache
    key = (As[0].device,) + tuple((a.data_ptr(), tuple(a.shape), a.dtype, a.is_contiguous(), a.device,
                                   b.data_ptr(), tuple(b.shape), b.dtype, b.is_contiguous(), b.device,
                                   float(al), float(p)) for a, b, al, p in zip(As, Bs, alphas, ps))
    st = _SETS.get(key)
    if st is None:
        st = _SETS[key] = _AdapterSet(As, Bs, alphas, ps)
        while len(_SETS) > _SETS_MAX:
            _SETS.popitem(last=False)
    else:
        _SETS.move_to_end(key)
    return st


class MultiLoraLinearFunction(torch.autograd.Function):
    """Mixed-adapter batch: rows [seg_off[s], seg_off[s+1]) of X (m x k) use
    adapter seg_adapter[s]; the adapters come as A0, B0, A1, B1, ... and each
    gets its gradients summed over its rows (papers.chlience.com notes, section
    5 "FusedMultiLoRA").  After them X's rows saved in 8 bits may follow, which
    the backward then keeps instead of X."""

    @staticmethod
    def forward(ctx, X, W, seg_off, seg_adapter, alphas, ps, seed: int, offset: int, *AB):
        *AB, X8 = AB if len(AB) % 2 else (*AB, None)
        As, Bs = AB[0::2], AB[1::2]
        kept = _input_tensors(X, X8)
        st = _adapter_set(As, Bs, alphas, ps)
        Y, S, keep = _of(W, "multi_lora_linear_fwd")(X, W, st.table, st.num, seg_off, seg_adapter, st.r_max, seed, offset)
        # the table holds A's and B's addresses alone: saved, they are guarded against changes, and kept here
        # they live on where a hook packs saved tensors away
        held = _weight_tensors(W)
        ctx.save_for_backward(seg_off, seg_adapter, S, keep, *kept, *held, *AB)
        ctx.adapter_set, ctx.kept, ctx.held, ctx.adapters = st, len(kept), len(held), AB
        ctx.group = getattr(W, "group", 0)
        return Y

    @staticmethod
    def backward(ctx, dY):
        seg_off, seg_adapter, S, keep, *rest = ctx.saved_tensors
        st = ctx.adapter_set
        W = _weight_again(rest[ctx.kept:ctx.kept + ctx.held], st.k, st.n, ctx.group)
        if ctx.kept == 1:
            bwd, X = _of(W, "multi_lora_linear_bwd"), rest[0]
        else:
            bwd, X = mxint8.multi_lora_mxint8_linear_bwd, Mxint8Input(*rest[:2], st.k)
        dAs, dBs = st.gradient_buffers()
        dX = bwd(dY.contiguous(), X, W, st.table, st.num, seg_off, seg_adapter, S, keep, st.r_max,
                 want_dX=ctx.needs_input_grad[0])
        grads = []
        for da, db in zip(dAs, dBs):
            grads += [da, db]
        return (dX, None, None, None, None, None, None, None, *grads, *[None] * (ctx.kept - 1))


def multi_lora_linear(X, W, seg_off, seg_adapter, As, Bs, alphas, ps, seed: int = 0, offset: int = 0, X8=None):
    """The layer over a mixed-adapter batch as an autograd function.  X8
    (lora_mxint8_quantize of X) is what the backward keeps in X's place."""
    AB = [t for pair in zip(As, Bs) for t in pair]
    kept = [] if X8 is None else [X8]
    return MultiLoraLinearFunction.apply(X, W, seg_off, seg_adapter, list(alphas), list(ps), seed, offset, *AB, *kept)


class LoraLinear(torch.nn.Module):
    """A frozen k x n weight, a tensor (kept in bf16), an Mxfp4Weight or an
    Int4Weight, with one LoRA adapter (A k x r, B r x n; B starts at zero).
    Dropout draws from the library's counter-based generator under this module's
    own seed; each training call advances the counter past the elements it used,
    so successive calls get fresh masks and a rerun from the same state reproduces
    them.  In eval mode dropout is off.

    save_bits = 8: a call that a backward may follow keeps its input in 8 bits
    (MXINT8) for it, and not the bf16 one.  Modules that share an input can share
    its 8-bit copy, made once: X8, lora_mxint8_quantize of the input's rows."""

    def __init__(self, weight, r: int, alpha: float, p: float = 0.0, seed: int = 0, save_bits: int = 16):
        super().__init__()
        if save_bits not in (8, 16):
            raise ValueError(f"save_bits = {save_bits} must be 8 or 16")
        self.k, self.n = k, n = weight.shape
        self.group = getattr(weight, "group", 0)
        self.save_bits = int(save_bits)
        if isinstance(weight, (Mxfp4Weight, Int4Weight)):
            self.register_buffer("weight_codes", weight.codes)
            self.register_buffer("weight_scales", weight.scales)
        else:
            self.register_buffer("weight", weight.detach().to(torch.bfloat16).contiguous())
        gen = torch.Generator(device="cpu").manual_seed(seed)
        a = torch.randn(k, r, generator=gen) / k ** 0.5
        self.A = torch.nn.Parameter(a.to(device=weight.device, dtype=torch.bfloat16))
        self.B = torch.nn.Parameter(torch.zeros(r, n, device=weight.device, dtype=torch.bfloat16))
        self.alpha, self.p, self.seed = float(alpha), float(p), int(seed)
        self.offset = 0  # next unused dropout counter (a multiple of 8)

    def forward(self, X: torch.Tensor, X8=None) -> torch.Tensor:
        wanted = X.requires_grad or self.A.requires_grad or self.B.requires_grad
        if X8 is None and self.save_bits == 8 and wanted and torch.is_grad_enabled():
            X8 = mxint8.lora_mxint8_quantize(X.detach().reshape(-1, X.shape[-1]).contiguous())
        p = self.p if self.training else 0.0
        offset = self.offset
        if p > 0.0:
            used = X.numel() // X.shape[-1] * X.shape[-1]
            self.offset += (used + 7) // 8 * 8
        held = (self.weight_codes, self.weight_scales) if hasattr(self, "weight_codes") else (self.weight,)
        W = _weight_again(held, self.k, self.n, self.group)
        return LoraLinearFunction.apply(X, W, self.A, self.B, self.alpha, p, self.seed, offset, X8)
