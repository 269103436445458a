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


# ---- a refused step ------------------------------------------------------------------------------

def everything(opt):
    """The optimizer's state and parameters, copied."""
    held = {id(p): {k: (x.clone() if isinstance(x, torch.Tensor) else x) for k, x in st.items()}
            for p, st in opt.state.items()}
    return held, [p.detach().clone() for g in opt.param_groups for p in g["params"]]


def same(a, b):
    assert a[0].keys() == b[0].keys()
    for p, st in a[0].items():
        assert st.keys() == b[0][p].keys()
        for name, x in st.items():
            y = b[0][p][name]
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)) if isinstance(x, torch.Tensor) else x == y, name
    assert all(torch.equal(x, y) for x, y in zip(a[1], b[1]))


def bad_type(opt, p):
    p.data = p.data.to(torch.float16)
    p.grad = torch.ones_like(p)


def bad_size(opt, p):
    p.grad = None
    p.data = p.data[:-1].clone()
    p.grad = torch.ones_like(p)


def bad_layout(opt, p):
    p.grad = None
    p.data = torch.zeros(14, dtype=p.dtype)[::2]
    p.grad = torch.ones(7, dtype=p.dtype)


def bad_gradient(opt, p):
    p.grad = torch.ones_like(p).to_sparse()


def shared_memory(opt, p):
    p.data = opt.param_groups[1]["params"][1].data[3:10]
    p.grad = torch.ones_like(p)


def bad_rate(opt, p):
    opt.param_groups[1]["lr"] = float("nan")


def bad_decay(opt, p):
    opt.param_groups[1]["weight_decay"] = float("inf")


def bad_betas(opt, p):
    opt.param_groups[1]["betas"] = (0.9, 1.0)


def bad_eps(opt, p):
    opt.param_groups[1]["eps"] = -1.0


def bad_seed(opt, p):
    opt.param_groups[1]["seed"] = "x"


def counter_elsewhere(opt, p):
    opt.param_groups[1]["capturable"] = not opt.param_groups[1]["capturable"]


SPOILERS = [bad_type, bad_size, bad_layout, bad_gradient, shared_memory, bad_rate, bad_decay, bad_betas, bad_eps, bad_seed,
            counter_elsewhere]


# (before the first step there is no size and no kind of count to differ from)
@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("before,spoil", [(steps, f) for steps in (0, 2) for f in SPOILERS
                                          if steps or f not in (bad_size, counter_elsewhere)])
def test_a_refused_step_changes_nothing(launches, spoil, capturable, before):
    # the second group's first parameter, or its numbers, are at fault: the first group is not stepped either,
    # no state is made and no count moves
    a, b = parameters(), parameters((7, 40))
    opt = lf.LoraAdamW([dict(params=a), dict(params=b)], capturable=capturable)
    for _ in range(before):
        opt.step()
    made = len(launches)
    spoil(opt, b[0])
    kept = everything(opt)
    for _ in range(2):
        with pytest.raises(Exception):
            opt.step()
        same(kept, everything(opt))
    assert len(launches) == made


def test_a_parameter_on_the_host_is_refused_before_it_gets_state(launches, monkeypatch):
    a, b = parameters(), parameters()
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: -1 if self is b[1] else 0)
    opt = lf.LoraAdamW([dict(params=a), dict(params=b)])
    for _ in range(2):
        with pytest.raises(ValueError, match="GPU"):
            opt.step()
        assert not opt.state and not launches
    # moved, it takes its first step
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    opt.step()
    assert [kw["step"] for _, kw in launches] == [1, 1]


def test_steps_and_counters_advance_once_a_step(launches):
    a, b = parameters(), parameters((5, 6, 7))
    opt = lf.LoraAdamW([dict(params=a, capturable=True), dict(params=b)])
    for t in range(1, 4):
        b[1].grad = None if t == 2 else torch.ones_like(b[1])
        opt.step()
        assert int(opt.state[a[0]]["step"]) == t and opt.state[a[0]]["step"] is opt.state[a[1]]["step"]
        assert [opt.state[p]["step"] for p in b] == [t, t - (t >= 2), t]
    # parameters whose steps differ have a call each
    assert [len(table.records) for table, _ in launches] == [2, 3, 2, 2, 2, 2, 1]
    spans = sorted((opt.state[p]["offset"], p.numel()) for p in a + b)
    assert all(x + n <= y for (x, n), (y, _) in zip(spans, spans[1:]))


def test_a_tensor_of_too_many_values_is_refused(monkeypatch):
    many = torch.zeros(1).expand(adamw.MOST + 1)
    with pytest.raises(ValueError, match="values, more than"):
        lf.adamw_table([many], [many], [many], [many])


@pytest.mark.parametrize("offsets,said", [([8], "one per parameter"), ([0, -8], "offsets"), ([0, 4], "multiple of 8"),
                                          ([0, 1 << 64], "offsets"), (np.array([0, -8]), "offsets")])
def test_offsets_are_checked(offsets, said):
    z = [torch.zeros(8) for _ in range(8)]
    with pytest.raises(ValueError, match=said):
        lf.adamw_table(z[:2], z[2:4], z[4:6], z[6:], offsets=offsets)


# ---- a captured step -----------------------------------------------------------------------------

def capture(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)


def test_a_first_step_is_not_captured(launches, monkeypatch):
    # its replays would make the state anew each time: moments of zero, step 1, the parameter as master
    ps = parameters()
    opt = lf.LoraAdamW(ps[:1], capturable=True)
    opt.step()
    opt.param_groups[0]["params"].append(ps[1])
    kept = everything(opt)
    capture(monkeypatch)
    with pytest.raises(ValueError, match="first step"):
        opt.step()
    same(kept, everything(opt))
    ps[1].grad = None
    opt.step()
    assert len(launches) == 2 and ps[1] not in opt.state


def test_a_step_counted_on_the_host_is_not_captured(launches, monkeypatch):
    ps = parameters()
    opt = lf.LoraAdamW(ps)
    opt.step()
    capture(monkeypatch)
    with pytest.raises(ValueError, match="capturable"):
        opt.step()
    assert len(launches) == 1 and opt.state[ps[0]]["step"] == 1


@pytest.mark.gpu
def test_a_refused_capture_leaves_the_optimizer_usable():
    p = torch.nn.Parameter(torch.ones(300, device="cuda", dtype=torch.bfloat16))
    opt = lf.LoraAdamW([p], lr=1e-2, capturable=True)
    p.grad = torch.ones_like(p)
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(ValueError, match="first step"):
            opt.step()
    assert not opt.state
    opt.step()
    graph2 = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph2):
        opt.step()
    for rep in range(3):
        graph2.replay()
        torch.cuda.synchronize()
        assert int(opt.state[p]["step"]) == rep + 2


# ---- autograd ------------------------------------------------------------------------------------

def test_autograd_sees_a_step(launches):
    ps = parameters()
    opt = lf.LoraAdamW(ps)
    ps[1].grad = None
    squares = [p.square().sum() for p in ps]
    versions = [p._version for p in ps]
    opt.step()
    assert [p._version > v for p, v in zip(ps, versions)] == [True, False]
    with pytest.raises(RuntimeError, match="inplace"):
        squares[0].backward()
    squares[1].backward()


@pytest.mark.gpu
@pytest.mark.parametrize("capturable", [False, True])
def test_a_backward_from_before_a_step_is_refused(capturable):
    W = torch.randn(72, 40, device="cuda").bfloat16()
    layer = lf.LoraLinear(W, 8, 2.0)
    opt = lf.LoraAdamW(layer.parameters(), capturable=capturable)
    X = torch.randn(5, 72, device="cuda").bfloat16().requires_grad_()
    layer(X).sum().backward()
    stale = layer(X).sum()
    opt.step()
    with pytest.raises(RuntimeError, match="inplace"):
        stale.backward()
    layer(X).sum().backward()  # and one from after it runs
    opt.step()


# ---- hyperparameters -----------------------------------------------------------------------------

@pytest.mark.parametrize("eps", [1e-40, 2.0 ** -127, -1.0, float("nan")])
def test_epsilons_that_the_library_refuses_are_refused_at_once(eps):
    with pytest.raises(ValueError, match="eps"):
        lf.LoraAdamW(parameters(), eps=eps)
