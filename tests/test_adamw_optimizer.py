"""What LoraAdamW hands to the library, on CPU tensors with the launch replaced: the
tables' contents, and what a step leaves behind when it is refused."""
import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as lf
from lora_fine_tuning_amd import adamw

F8 = torch.float8_e4m3fn


@pytest.fixture
def launches(monkeypatch):
    """(table, keywords) of every call that a step makes; the tensors pass for a GPU's."""
    made = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(adamw, "lora_adamw_step", lambda table, **kw: made.append((table, kw)))
    return made


def parameters(sizes=(40, 7), dtype=torch.bfloat16):
    ps = [torch.nn.Parameter(torch.ones(n, dtype=dtype)) for n in sizes]
    for p in ps:
        p.grad = torch.ones_like(p)
    return ps


def column(tensors):
    return [t.data_ptr() for t in tensors]


def check_table(table, opt, ps):
    """Every address is that of the state's tensor of now, and the moments' width is theirs."""
    rec, states = table.records, [opt.state[p] for p in ps]
    bits = {F8: 8, torch.float32: 32}[states[0]["m"].dtype]
    assert all(st[x].dtype == states[0]["m"].dtype for st in states for x in "mv")
    assert table.state_bits == bits
    names = ["m", "v"] + (["m_scale", "v_scale"] if bits == 8 else []) + (["master"] if "master" in states[0] else [])
    cols = dict(m=adamw._M, v=adamw._V, m_scale=adamw._M_SCALE, v_scale=adamw._V_SCALE, master=adamw._MASTER)
    for name, col in cols.items():
        want = column(st[name] for st in states) if name in names else [0] * len(ps)
        assert rec[:, col].tolist() == want, name
    assert rec[:, adamw._PARAM].tolist() == column(ps)
    assert rec[:, adamw._GRAD].tolist() == column(p.grad for p in ps)
    assert rec[:, adamw._N].tolist() == [p.numel() for p in ps]


@pytest.mark.parametrize("first,then", [(8, 32), (32, 8)])
@pytest.mark.parametrize("master", [True, False])
def test_moments_of_another_width_after_a_cleared_state(launches, first, then, master):
    ps = parameters()
    opt = lf.LoraAdamW(ps, state_bits=first, master=master)
    opt.step()
    check_table(launches[-1][0], opt, ps)
    opt.state.clear()
    opt.param_groups[0]["state_bits"] = then
    opt.step()
    assert launches[-1][0].state_bits == then and len(launches) == 2
    check_table(launches[-1][0], opt, ps)


def test_a_group_that_takes_anothers_place(launches):
    a, b = parameters(), parameters()
    opt = lf.LoraAdamW([dict(params=a, state_bits=8), dict(params=b, state_bits=32)])
    opt.step()
    del opt.param_groups[0]
    opt.step()
    assert [table.state_bits for table, _ in launches] == [8, 32, 32]
    check_table(launches[-1][0], opt, b)


def test_moments_of_both_widths_in_a_group(launches):
    # a parameter that joins after the group's width was changed: each width has a call of its own
    a, b = parameters((40,)), parameters((7,))
    opt = lf.LoraAdamW(a, state_bits=8)
    opt.step()
    opt.param_groups[0]["state_bits"] = 32
    opt.param_groups[0]["params"] += b
    opt.step()
    assert sorted(table.state_bits for table, _ in launches[1:]) == [8, 32]
    for table, _ in launches[1:]:
        check_table(table, opt, a if table.state_bits == 8 else b)


def test_state_that_was_replaced_is_read_anew(launches, monkeypatch):
    ps = parameters()
    opt = lf.LoraAdamW(ps)
    opt.step()
    for st in opt.state.values():
        for name in ("m", "v", "m_scale", "v_scale", "master"):
            st[name] = st[name].clone()
    opt.step()
    check_table(launches[-1][0], opt, ps)
    # moved to the host and not back: refused, as in the first step
    opt.state[ps[1]]["v"] = away = opt.state[ps[1]]["v"].clone()
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: -1 if self is away else 0)
    with pytest.raises(ValueError, match="GPU"):
        opt.step()
    # two parameters that came to share memory
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    both = torch.zeros(47, dtype=torch.bfloat16)
    ps[0].data, ps[1].data = both[:40], both[38:45]
    with pytest.raises(ValueError, match="share memory"):
        opt.step()
