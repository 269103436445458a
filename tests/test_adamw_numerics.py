"""The AdamW step's arithmetic where single roundings add up: many steps' worth of small
decays, epsilons at the end of fp32's range, corrections formed on the device.  References in 64 bits from the formulas."""
import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as lf
from parity import log


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("master", [True, False])
@pytest.mark.parametrize("lr,wd", [(1e-3, 1e-2), (1e-4, 1e-2), (1e-5, 1e-2), (2e-6, 1e-2), (1e-6, 1e-2)])
@pytest.mark.parametrize("n", [1 << 18, (1 << 18) + 777])
def test_small_decays_are_not_lost(lr, wd, master, n):
    # w in [1/2, 1), where fp32's step is 2^-24, and updates of both signs far larger than a step: each w is
    # rounded by an even draw from half a step up and down, 2^-24 / sqrt(12) as a standard deviation.  Over n
    # values the mean is off by 5 / sqrt(n) of that, and by the decay's and the update's own roundings:
    # 2^-23 of the mean decay, and of the update m / sqrt(v) (2^-20 with its root, quotient and products, of
    # mixed signs) no more than 2^-20 of its mean over 1
    log(f"lr={lr} wd={wd} master={master} n={n}")
    g = torch.Generator().manual_seed(int(lr * 1e7))
    w = 0.5 + 0.5 * torch.rand(n, generator=g)
    grad = torch.randn(n, generator=g)
    m, v = 0.3 * torch.randn(n, generator=g), 0.5 + torch.rand(n, generator=g)
    param = w.bfloat16().cuda() if master else w.cuda()
    held = w.cuda() if master else param
    ms, vs = m.cuda(), v.cuda()
    table = lf.adamw_table([param], [grad.cuda()], [ms], [vs], masters=[held] if master else None)
    lf.lora_adamw_step(table, lr=lr, weight_decay=wd, step=50)
    torch.cuda.synchronize()
    m2, v2 = 0.9 * f64(m) + 0.1 * f64(grad), 0.999 * f64(v) + 0.001 * f64(grad) ** 2
    up = lr * m2 / (1 - 0.9 ** 50) / (np.sqrt(v2 / (1 - 0.999 ** 50)) + 1e-8)
    want = f64(w) - lr * wd * f64(w) - up
    bound = 5 * 2.0 ** -24 / np.sqrt(12 * n) + 2.0 ** -23 * lr * wd + 2.0 ** -20 * (lr * 5 / np.sqrt(n) + abs(up.mean()))
    off = (f64(held) - want).mean()
    assert abs(off) <= bound, (off, bound, lr * wd * f64(w).mean())
    if lr * wd <= 1e-7:  # the bound is a small part of the decay itself
        assert bound < 0.02 * lr * wd


@pytest.mark.gpu
def test_infinite_parameters_stay_infinite():
    for n in (2048, 300):
        for wd in (0.0, 0.1):
            w = torch.ones(n, device="cuda")
            w[3], w[5], w[7] = float("inf"), -float("inf"), float("nan")
            z = [torch.zeros(n, device="cuda") for _ in range(2)]
            lf.lora_adamw_step(lf.adamw_table([w], [torch.ones(n, device="cuda")], z[:1], z[1:]), lr=1e-2,
                               weight_decay=wd, step=1)
            torch.cuda.synchronize()
            assert w[3] == float("inf") and w[5] == -float("inf") and torch.isnan(w[7])
            assert torch.isfinite(w).sum() == n - 3


def test_subnormal_epsilons_are_refused():
    import os

    from lora_fine_tuning_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    lib = _lib.load()

    def call(eps):
        return lib.lora_adamw_step(None, 0, 1, 1, 8, 1e-3, 0.9, 0.999, eps, 0.0, 1, None, 0, None)

    for eps in (1e-40, 1e-300, 2.0 ** -127, float(np.nextafter(2.0 ** -126, 0))):
        assert call(eps) == -1, eps
        assert b"eps" in lib.lora_last_error_message()
    for eps in (0.0, 2.0 ** -126, 1e-8, 1.0):
        assert call(eps) == 0, eps


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2048, 300])
@pytest.mark.parametrize("bits", [8, 32])
def test_a_parameter_without_gradients_so_far(n, bits):
    # moments of zero and a gradient of zero (an adapter's A while B is zero): only the decay moves w, down to
    # the smallest eps, and eps = 0 is 0 / 0
    F8 = torch.float8_e4m3fn
    for eps in (2.0 ** -126, 1e-8, 0.0):
        w, g = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
        m, v = (torch.zeros(n, dtype=torch.uint8 if bits == 8 else torch.float32, device="cuda") for _ in range(2))
        scales = [torch.zeros(-(-n // 256), device="cuda") for _ in range(2)]
        kw = dict(m_scales=scales[:1], v_scales=scales[1:]) if bits == 8 else {}
        table = lf.adamw_table([w], [g], [m.view(F8) if bits == 8 else m], [v.view(F8) if bits == 8 else v], **kw)
        lf.lora_adamw_step(table, lr=0.5, weight_decay=0.25, eps=eps, step=1)
        torch.cuda.synchronize()
        assert (w == 0.875).all() if eps else torch.isnan(w).all()
        assert not m.any() and not v.any()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_replays_follow_the_formulas(bits):
    # a captured step against the reference of the plain one, replay by replay
    from test_adamw import HYPER, Tensors
    lr, wd, E = HYPER["lr"], HYPER["weight_decay"], 2.0 ** -24
    T = Tensors([700, 5000], bits, torch.bfloat16, torch.bfloat16, True, seed=6)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run():
        counter.add_(1)
        lf.lora_adamw_step(T.table, step_dev=counter, seed=4, **HYPER)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep in range(3):
        for i, grad in enumerate(T.g):
            grad.copy_(torch.randn(grad.numel(), generator=torch.Generator().manual_seed(rep * 10 + i)))
        torch.cuda.synchronize()
        before = [T.before(i) for i in range(2)]
        graph.replay()
        torch.cuda.synchronize()
        t = int(counter)
        assert t == rep + 2
        # 1 - beta^t is formed on the device from fp32 logarithms (2^-23 of themselves) and t: the exponent is off
        # by 2^-22 of itself, and 1 - beta^t, at least half of t |ln beta| here, by 2^-21 of itself at most; with the
        # root half of that, and the quotient, the update moves by 2^-20 of itself
        for (w, g, m, v), master in zip(before, T.master):
            m2, v2 = 0.9 * m + 0.1 * g, 0.999 * v + 0.001 * g * g
            rate = lr / (1 - 0.9 ** t) / (np.sqrt(v2 / (1 - 0.999 ** t)) + 1e-8)
            want = w - lr * wd * w - rate * m2
            slack = 4 * E * np.abs(w) + (2.0 ** -20 + 24 * E) * rate * np.abs(m2) + 8 * E * rate * (np.abs(m) + np.abs(g))
            assert (np.abs(f64(master) - want) <= slack).all()
