"""AdamW over many tensors in one call, with moments in 8 or 32 bits.

`lora_adamw_step` has the name of its C-ABI entry point in include/lora_fused.h
and works on an `adamw_table`; `LoraAdamW` is a torch optimizer over it."""
from __future__ import annotations

from typing import Optional, Sequence

import numpy as np
import torch

from ._lib import _check, _elsewhere, _handle, _on_device, load

BLOCK = 256  # values that share a scale of the 8-bit moments
MOST = ((1 << 24) - 1) * 2048  # values of one tensor (a launch's work-groups, 2048 values each)
_PARAM, _GRAD, _MASTER, _M, _V, _M_SCALE, _V_SCALE, _N, _OFFSET = range(9)


class AdamwTable:
    """The records of one call (mirrors of lora_adamw_tensor, 72 bytes each) and
    the tensors they point into, which stay alive with it."""

    def __init__(self, records, tensors, device, param_bf16: bool, grad_bf16: bool, state_bits: int):
        self.records, self.tensors, self.device = records, tensors, device
        self.address = records.ctypes.data
        self.param_bf16, self.grad_bf16, self.state_bits = param_bf16, grad_bf16, state_bits


def _column(ts: Sequence[torch.Tensor], name: str, count: int, dtypes, numels=None):
    """Their addresses, after the checks that every tensor of the column shares."""
    if len(ts) != count:
        raise ValueError(f"{name} must have one tensor per parameter ({count}), got {len(ts)}")
    dtype = ts[0].dtype if count else dtypes[0]
    if dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {dtype}")
    if {t.dtype for t in ts} - {dtype}:
        i = next(i for i, t in enumerate(ts) if t.dtype != dtype)
        raise TypeError(f"{name}[{i}] is {ts[i].dtype}, {name}[0] {dtype}")
    if not all(map(torch.Tensor.is_contiguous, ts)):
        raise ValueError(f"{name}[{next(i for i, t in enumerate(ts) if not t.is_contiguous())}] must be contiguous")
    if numels is not None and list(map(torch.Tensor.numel, ts)) != numels:
        i = next(i for i, t in enumerate(ts) if t.numel() != numels[i])
        raise ValueError(f"{name}[{i}] must have {numels[i]} values, got {ts[i].numel()}")
    return np.fromiter(map(torch.Tensor.data_ptr, ts), np.uint64, count), dtype


def _apart(records, widths) -> None:
    """Refuse records that share memory which a step writes."""
    spans = []
    n = records[:, _N].astype(np.int64)
    for col, width in widths:
        size = -(-n // BLOCK) * 4 if col in (_M_SCALE, _V_SCALE) else n * width
        at = records[:, col].astype(np.int64)
        spans.append(np.stack([at, at + size], 1)[size > 0])
    s = np.concatenate(spans)
    s = s[np.argsort(s[:, 0], kind="stable")]
    if (s[1:, 0] < s[:-1, 1]).any():
        raise ValueError("two of the tensors that a step writes share memory")


def adamw_table(params, grads, ms, vs, *, m_scales=None, v_scales=None, masters=None,
                offsets: Optional[Sequence[int]] = None) -> AdamwTable:
    """The records of lora_adamw_step for these tensors: params fp32 or bf16,
    grads fp32 or bf16, and moments as float32, or as float8_e4m3fn with m_scales
    and v_scales of one float32 for each 256 values.  masters: fp32 copies of
    bf16 params.  offsets: each tensor's first counter of the random roundings
    (a multiple of 8; by default the tensors follow one another)."""
    params, grads, ms, vs = list(params), list(grads), list(ms), list(vs)
    count = len(params)
    if count == 0:
        raise ValueError("params must not be empty")
    device = params[0].device
    numels = list(map(torch.Tensor.numel, params))
    if max(numels) > MOST:
        raise ValueError(f"params[{numels.index(max(numels))}] has {max(numels)} values, more than {MOST}")
    held8 = ms[0].dtype == torch.float8_e4m3fn if ms else False
    moment = (torch.float8_e4m3fn,) if held8 else (torch.float32,)
    f32, either = (torch.float32,), (torch.float32, torch.bfloat16)
    rec = np.zeros((count, 9), dtype=np.uint64)
    rec[:, _PARAM], pt = _column(params, "params", count, either)
    rec[:, _GRAD], gt = _column(grads, "grads", count, either, numels)
    rec[:, _M], _ = _column(ms, "ms", count, moment, numels)
    rec[:, _V], _ = _column(vs, "vs", count, moment, numels)
    tensors = [params, grads, ms, vs]
    widths = [(_PARAM, 2 if pt == torch.bfloat16 else 4), (_M, 1 if held8 else 4), (_V, 1 if held8 else 4)]
    if held8:
        blocks = [-(-e // BLOCK) for e in numels]
        for col, ts, name in ((_M_SCALE, m_scales, "m_scales"), (_V_SCALE, v_scales, "v_scales")):
            if ts is None:
                raise ValueError("8-bit moments need m_scales and v_scales")
            rec[:, col], _ = _column(list(ts), name, count, f32, blocks)
            tensors.append(list(ts))
            widths.append((col, 4))
    elif m_scales is not None or v_scales is not None:
        raise ValueError("m_scales and v_scales go with float8_e4m3fn moments")
    if masters is not None:
        if pt != torch.bfloat16:
            raise ValueError("master copies go with bf16 params")
        rec[:, _MASTER], _ = _column(list(masters), "masters", count, f32, numels)
        tensors.append(list(masters))
        widths.append((_MASTER, 4))
    if offsets is None:
        padded = [(e + 7) // 8 * 8 for e in numels]
        offsets = np.concatenate([[0], np.cumsum(padded)[:-1]])
    elif len(offsets) != count or min(offsets) < 0 or max(offsets) >= 1 << 64:
        raise ValueError(f"offsets must be one per parameter ({count}), each in [0, 2^64)")
    rec[:, _N], rec[:, _OFFSET] = numels, offsets
    if (rec[:, _OFFSET] & np.uint64(7)).any():
        raise ValueError("each offset must be a multiple of 8")
    # the device last, so that host tests can reach every other check with CPU tensors
    index = params[0].get_device()
    for ts in tensors:
        places = list(map(torch.Tensor.get_device, ts))
        if index < 0 or places.count(index) != len(places):
            other = next((t for t, i in zip(ts, places) if i < 0 or i != index), ts[0])
            raise ValueError(f"a tensor is on {other.device}: all must be on one GPU ({device})")
    _apart(rec, widths)
    return AdamwTable(rec, tensors, device, pt == torch.bfloat16, gt == torch.bfloat16, 8 if held8 else 32)


def lora_adamw_step(table: AdamwTable, *, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                    weight_decay: float = 0.0, step: int = 0, step_dev: Optional[torch.Tensor] = None, seed: int = 0,
                    stream=None) -> None:
    """One step (the step-th, from 1; or the one whose number the int64 device
    tensor step_dev holds) over the table's tensors, in place.  Autograd does not
    see the change (torch.autograd.graph.increment_version tells it; LoraAdamW does)."""
    if _elsewhere(table.device, stream):
        with _on_device(table.device, stream):
            return lora_adamw_step(table, lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay,
                                   step=step, step_dev=step_dev, seed=seed)
    if step_dev is not None:
        _need_counter(step_dev, table.device)
        step_dev = step_dev.data_ptr()
    _check(load().lora_adamw_step(table.address, len(table.records), table.param_bf16, table.grad_bf16,
                                  table.state_bits, lr, beta1, beta2, eps, weight_decay, step, step_dev,
                                  seed % (1 << 64), _handle(table.device)))


def _need_counter(counter: torch.Tensor, device) -> None:
    if counter.dtype != torch.int64 or counter.numel() != 1 or counter.device != device:
        raise ValueError(f"step_dev must be one int64 on {device}")


def _hyper_allowed(lr, beta1, beta2, eps, weight_decay, seed) -> None:
    """The library's own checks of a step's numbers, by a call on no tensors."""
    _check(load().lora_adamw_step(None, 0, 0, 0, 32, lr, beta1, beta2, eps, weight_decay, 1, None, seed % (1 << 64), None))


class LoraAdamW(torch.optim.Optimizer):
    """AdamW (decoupled weight decay) for adapter tensors, all of a group in one
    call of the library.

    state_bits: 8 or 32, the bits of a moment.  master: bf16 parameters get an
    fp32 copy that is updated in their place (a bf16 loses updates below half of
    its last place).  seed: of the 8-bit moments' random rounding.  capturable:
    the step number lives on the device, so that a captured step() counts on in
    every replay; the group's learning rate and decay are those of the capture.
    A step is captured with it only, and after each parameter's first one, which
    makes its state.

    Parameters are contiguous GPU tensors, fp32 or bf16.  A parameter without a
    gradient is left out of a step (the shared counter of a capturable group goes
    on).  A parameter whose values are replaced from outside keeps its master copy
    until its state is cleared."""

    def __init__(self, params, lr: float = 1e-4, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.0,
                 state_bits: int = 8, master: bool = True, seed: int = 0, capturable: bool = False):
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits = {state_bits} must be 8 or 32")
        if not lr >= 0.0 or not weight_decay >= 0.0 or not eps >= 0.0:
            raise ValueError(f"lr = {lr}, weight_decay = {weight_decay} and eps = {eps} must be >= 0")
        if 0.0 < eps < 2.0 ** -126:
            raise ValueError(f"eps = {eps} must be 0 or at least 2^-126")
        if not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError(f"betas = {betas} must be in [0, 1)")
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay,
                                      state_bits=state_bits, master=master, seed=seed, capturable=capturable))

    def _counter(self, group, device) -> torch.Tensor:
        """The step counter that a captured group's parameters on a device share."""
        for p in group["params"]:
            at = self.state[p].get("step") if p in self.state else None
            if isinstance(at, torch.Tensor) and at.device == device:
                return at
        return torch.zeros(1, dtype=torch.int64, device=device)

    @staticmethod
    def _new_state(p: torch.Tensor, group, step, offset: int) -> dict:
        n, dev = p.numel(), p.device
        st = {"step": step, "offset": offset}
        if group["state_bits"] == 8:
            st["m"], st["v"] = (torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
                                for _ in range(2))
            st["m_scale"], st["v_scale"] = (torch.zeros((n + BLOCK - 1) // BLOCK, device=dev) for _ in range(2))
        else:
            st["m"], st["v"] = (torch.zeros(n, dtype=torch.float32, device=dev) for _ in range(2))
        if group["master"] and p.dtype == torch.bfloat16:
            st["master"] = p.detach().reshape(-1).float()
        return st

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        calls, fresh, counters = self._calls()  # refuses before anything has changed
        self.state.update(fresh)
        for counter in counters:
            counter.add_(1)
        for table, ps, states, t, hyper in calls:
            if isinstance(t, torch.Tensor):
                lora_adamw_step(table, step_dev=t, **hyper)
            else:
                for st in states:
                    st["step"] = t
                lora_adamw_step(table, step=t, **hyper)
            # a backward through a graph from before the step is refused, as after any in-place change
            torch.autograd.graph.increment_version(ps)
        return loss

    def _calls(self):
        """What a step does, with every check and no change: its calls, each a table,
        the parameters, their states and step (a number, or the counter on the device)
        and the hyperparameters; the states of parameters that have none; the counters."""
        calls, fresh, counters, shared = [], {}, {}, {}
        capturing = torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()
        end = None  # of the random rounding's counters that are taken
        for index, group in enumerate(self.param_groups):
            hyper = dict(lr=float(group["lr"]), beta1=group["betas"][0], beta2=group["betas"][1], eps=group["eps"],
                         weight_decay=group["weight_decay"], seed=group["seed"])
            on_device = bool(group["capturable"])
            kinds = {}  # the tensors of one call share a device, types and a step
            for p in group["params"]:
                g = p.grad
                if g is None:
                    continue
                if capturing and not on_device:
                    raise ValueError("a captured step needs capturable=True: its replays would repeat one step's number")
                st = self.state.get(p)
                if not st:
                    if capturing:
                        raise ValueError("a parameter's first step cannot be captured: every replay would begin "
                                         "with empty moments again (take a step before the capture)")
                    step = 0
                    if on_device:
                        step = shared.get((index, p.device))
                        if step is None:
                            step = shared[index, p.device] = self._counter(group, p.device)
                    if end is None:
                        end = max((st["offset"] + st["m"].numel() for st in self.state.values() if st), default=0)
                    st = fresh[p] = self._new_state(p, group, step, -(-end // BLOCK) * BLOCK)
                    end = st["offset"] + p.numel()
                t = st["step"]
                if isinstance(t, torch.Tensor) != on_device:
                    raise ValueError("capturable was changed after a parameter's first step (a loaded state follows it)")
                key = (p.get_device(), p.dtype, g.dtype, "master" in st, st["m"].dtype, id(t) if on_device else t)
                kinds.setdefault(key, []).append((p, g, st))
            if kinds:
                _hyper_allowed(**hyper)
            for members in kinds.values():
                ps, gs, states = map(list, zip(*members))
                t = states[0]["step"]
                calls.append((self._table(ps, gs, states), ps, states, t if on_device else t + 1, hyper))
                if on_device:
                    _need_counter(t, ps[0].device)
                    counters[id(t)] = t
        return calls, fresh, list(counters.values())

    @staticmethod
    def _table(ps, grads, states) -> AdamwTable:
        """The table of these parameters, made anew at each step: between two steps
        any tensor may have moved, and the state's may have been replaced."""
        if {g.layout for g in grads} != {torch.strided}:
            raise ValueError("gradients must be dense")
        if not all(map(torch.Tensor.is_contiguous, grads)):
            grads = [g.contiguous() for g in grads]
        each = lambda name: [st[name] for st in states] if name in states[0] else None  # noqa: E731
        try:
            return adamw_table(ps, grads, each("m"), each("v"), m_scales=each("m_scale"), v_scales=each("v_scale"),
                               masters=each("master"), offsets=each("offset"))
        except ValueError:
            for p, st in zip(ps, states):
                if p.numel() != st["m"].numel():
                    raise ValueError(f"a parameter had {st['m'].numel()} values when its moments were made, "
                                     f"now {p.numel()}") from None
            raise

    def load_state_dict(self, state_dict) -> None:
        """The moments keep their own types (torch's loader would cast them to
        the parameters')."""
        saved = state_dict["state"]
        super().load_state_dict(dict(state_dict, state={}))
        for group, old in zip(self.param_groups, state_dict["param_groups"]):
            for p, i in zip(group["params"], old["params"]):
                if i not in saved:
                    continue
                st = {name: x.to(device=p.device, copy=True) if isinstance(x, torch.Tensor) else x
                      for name, x in saved[i].items()}
                if group["capturable"]:  # one counter again
                    st["step"] = self._counter(group, p.device).copy_(torch.as_tensor(st["step"]))
                elif isinstance(st["step"], torch.Tensor):
                    st["step"] = int(st["step"])
                self.state[p] = st
