"""The gradient norm and the AdamW step at the edges of their number formats.
Helpers and bounds as in test_gpu_optim.
"""
import math

import numpy as np
import pytest
import torch

import ddp_bucketed_gradient_amd as D  # noqa: F401
from gpu_util import require_gpu, say
from test_gpu_optim import Case, f64, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("p,master", [("f32", False), ("bf16", False), ("f16", True)])
def test_an_element_does_not_depend_on_the_others(p, master):
    """Infinite, NaN and huge elements in one block of every four: all other
    blocks get the same bits as without them, parameters, codes and scales, and
    so do the other parameters of the block itself. Roots from 2^-94 to 2^30."""
    n = 64 * 300
    cases = []
    for special in (False, True):
        c = Case(p, "f32", "f8", master, numels=[n, 777], seed=80, step=5, random_seed=3)
        gen = torch.Generator(device="cuda").manual_seed(80)
        s = torch.randint(42, 148, (300,), generator=gen, device="cuda")
        s[::4] = 130
        c.opt.root_scale[0].view(torch.uint8).copy_(s)
        c.opt.exp_avg_root[0].view(torch.uint8).clamp_(min=8)
        g = torch.randn(n, generator=gen, device="cuda").view(300, 64) * torch.exp2(
            torch.randint(-60, 28, (300, 64), generator=gen, device="cuda").float())
        c.grads[0].copy_(g.view(-1))
        if special:
            for k, x in ((0, math.inf), (9, math.nan), (30, 1e30), (63, -math.inf)):
                c.grads[0].view(300, 64)[::4, k] = x
        c.opt.step(lr=1e-2)
        torch.cuda.synchronize()
        cases.append(c)
    a, b = (c.opt for c in cases)
    block = np.arange(300) % 4 != 0
    for ts, rows in ((a.exp_avg, b.exp_avg), (a.exp_avg_root, b.exp_avg_root), (a.avg_scale, b.avg_scale),
                     (a.root_scale, b.root_scale), (a.params[0], b.params[0])):
        x, y = (raw(t[0]).reshape(300, -1)[block] for t in (ts, rows))
        assert np.array_equal(x, y)
    x, y = (f64(o.params[0][0]).reshape(300, 64) for o in (a, b))
    other = np.ones(64, dtype=bool)
    other[[0, 9, 30, 63]] = False
    assert np.array_equal(x[:, other], y[:, other])
    if master:
        x, y = (f64(o.master[0]).reshape(300, 64)[:, other] for o in (a, b))
        assert np.array_equal(x, y)


@pytest.mark.parametrize("p,master", [("f32", False), ("bf16", True), ("f16", False)])
@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 2.0 ** -128, 2.0 ** -126, 2e-38])
def test_epsilons_around_the_smallest_normal_number(eps, zero, p, master):
    """0 / (0 + eps) is 0 for every eps > 0, 8-bit states included. In the other
    elements eps is below 2^-24 of r, so that its own rounding to fp32 (up to a
    half at 1e-45) does not show."""
    say(f"eps={eps} zero={zero} p={p}")
    c = Case(p, "f32", "f8", master, zero=True, seed=81, eps=eps)
    for _ in range(2):
        c.new_grads()
        if zero:
            for t in c.grads[1::2]:
                t.zero_()
            c.grads[10][64:200] = 0.0
        before = c.host()
        c.opt.step(lr=1e-2)
        c.check_step(before, 1e-2, 1.0, f"eps {eps}")


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_epsilon_zero_with_gradients_everywhere(state):
    c = Case("f32", "f32", state, zero=True, seed=82, eps=0.0)
    c.new_grads()
    before = c.host()
    c.opt.step(lr=1e-2)
    c.check_step(before, 1e-2, 1.0, "eps 0")
