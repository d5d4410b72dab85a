"""The gradient norm and the AdamW step at the edges of their number formats.
Helpers and bounds as in test_gpu_optim.
"""
import math

import numpy as np
import pytest
import torch

import ddp_bucketed_gradient_amd as D
from gpu_util import require_gpu, say
from oracle import optim as OO
from test_gpu_optim import Case, check_codes, f64, raw

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


def test_roots_around_the_underflow_of_their_squares():
    """Stored roots from 2^-110 to 2^-85 that decay without a gradient. From
    2^-95 on (where 2^64 v is a normal number) the new root is within the
    arithmetic's bound; below, it falls off gradually: never above the true one,
    at least 0.68 of it down to 2^-96 (the correction step of the root gives
    1.5 c - c^2 / 2 for c = r^2 2^190 where sqrt(c) is true: 0.6875 of it at c =
    1/4). Squares there are multiples of 2^-149, two roundings of half a step in
    c = 2^-23, which 1.5 2^-95 takes to 2^-117.4 in r."""
    first, last = 17, 42                                    # scales 2^(s - 127), codes from 2^-6 to 448
    n = 64 * (last - first + 1)
    c = Case("f32", "f32", "f8", numels=[n], zero=True, seed=83, betas=(0.9, 0.96), step=7, random_seed=5)
    codes = np.concatenate([np.arange(8, 72) + (s % 2) * 55 for s in range(first, last + 1)]).astype(np.uint8)
    scales = np.arange(first, last + 1).astype(np.uint8)
    c.opt.exp_avg_root[0].view(torch.uint8).copy_(torch.from_numpy(codes))
    c.opt.root_scale[0].view(torch.uint8).copy_(torch.from_numpy(scales))
    c.grads[0].zero_()
    r = OO.decode(codes, scales) * math.sqrt(0.96)
    c.opt.step(lr=1e-2)
    torch.cuda.synchronize()
    got_c, got_s = raw(c.opt.exp_avg_root[0]), raw(c.opt.root_scale[0])
    _, ur = OO.random16(5, 8, np.arange(n, dtype=np.uint64))
    for b in range(last - first + 1):
        cut = slice(64 * b, 64 * b + 64)
        if r[cut].min() >= 2.0 ** -95:
            check_codes(r[cut], 5 * OO.U * r[cut], ur[cut], True, got_c[cut], got_s[b:b + 1], f"block {b}")
    s = got_s.astype(np.int64)
    unit = np.repeat(np.ldexp(1.0, s - 127), 64)
    got = OO.CODES[got_c]
    high = r * (1 + 6 * OO.U) + 2.0 ** -117 + unit * 2.0 ** -30
    low = np.where(r >= 2.0 ** -95, r * (1 - 6 * OO.U), np.where(r >= 2.0 ** -96, 0.68 * r, 0.0)) - unit * 2.0 ** -30

    def at(y):
        lo, up, pos = OO.encode_levels(np.maximum(y, 0.0), s, ur, True)
        return np.where(pos >= 1, up, lo)
    assert (got <= at(high)).all() and (got >= at(low)).all()
    assert (got[r >= 2.0 ** -96] > 0).all()
    assert np.array_equal(raw(c.opt.exp_avg[0]) & 127, np.zeros(n, np.uint8))


def test_random_bits_where_a_tile_crosses_2_to_the_32_groups():
    """A second variable whose groups of four elements pass index 2^32 inside a
    tile: in its first wave, in the second group of a lane, and in a rest."""
    big, n1 = 1 << 34, 4096 + 1500
    need = (big + n1) * 6 + (8 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    new = lambda n, dt: torch.zeros(n, dtype=torch.uint8, device="cuda").view(dt)  # noqa: E731
    p0, g0 = new(2 * big, torch.bfloat16), new(2 * big, torch.bfloat16)
    m0, r0 = new(big, torch.float8_e4m3fn), new(big, torch.float8_e4m3fn)
    ms0, rs0 = new(big // 64, torch.float8_e8m0fnu), new(big // 64, torch.float8_e8m0fnu)
    gen = torch.Generator(device="cuda").manual_seed(86)
    for cross in (64, 2048 + 1088, 4096 + 1088):            # elements of variable 1 below 2^34
        say(f"2^32 groups reached at element {cross}")
        n0 = big - cross
        p = (torch.randn(n1, generator=gen, device="cuda") * 0.02).bfloat16()
        g = (torch.randn(n1, generator=gen, device="cuda") * 1e-3).bfloat16()
        opt = D.AdamW([p0[:n0], p], [g0[:n0], g], lr=1e-2, weight_decay=0.0, state="f8", seed=99, states={
            "exp_avg": [m0[:n0], new(n1, torch.float8_e4m3fn)], "exp_avg_root": [r0[:n0], new(n1, torch.float8_e4m3fn)],
            "avg_scale": [ms0[:-(-n0 // 64)], new(-(-n1 // 64), torch.float8_e8m0fnu)],
            "root_scale": [rs0[:-(-n0 // 64)], new(-(-n1 // 64), torch.float8_e8m0fnu)]})
        w0, gg = f64(p), f64(g)
        opt.step()
        torch.cuda.synchronize()
        (_, m, _, r), (_, bm, _, br) = OO.adamw(w0, gg, 0 * gg, 0 * gg, t=1, lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8,
                                                weight_decay=0.0, gscale=1.0)
        um, ur = OO.random16(99, 1, np.uint64(n0) + np.arange(n1, dtype=np.uint64))
        check_codes(m, bm, um, False, raw(opt.exp_avg[1]), raw(opt.avg_scale[1]), f"m, crossing at {cross}")
        check_codes(r, br, ur, True, raw(opt.exp_avg_root[1]), raw(opt.root_scale[1]), f"r, crossing at {cross}")
        opt.close()
        del opt
    del p0, g0, m0, r0, ms0, rs0
    torch.cuda.empty_cache()


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_a_norm_above_the_range_of_fp32_is_not_finite(state):
    """Finite gradients whose norm fp32 cannot hold: the norm that is reported is
    infinite, and a step that is to be skipped on such a norm is."""
    c = Case("f32", "f32", state, seed=85)
    c.new_grads()
    c.grads[9].fill_(3e38)
    n = D.GradNorm(c.grads)
    before = {k: s.bytes.cpu().numpy() for k, s in c.stores.items()}
    norm = n.compute(max_norm=1.0, skip_nonfinite=True)
    c.opt.step(lr=1e-2, clip=n)
    torch.cuda.synchronize()
    assert math.isinf(norm.item()) and n.skipped.item() == 1 and c.opt.steps_done == 0
    for k, s in c.stores.items():
        assert np.array_equal(before[k], s.bytes.cpu().numpy()), k
    n.compute(max_norm=1.0, grad_scale=2.0 ** -20, skip_nonfinite=True)      # in range again
    assert math.isfinite(norm.item()) and n.skipped.item() == 0
    n.compute(max_norm=1.0)                                                  # nobody asked to skip
    assert math.isinf(norm.item()) and n.skipped.item() == 0


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_gradients_that_are_not_finite_leave_nan(state):
    """An infinite gradient makes m and r infinite, their quotient is NaN; NaN
    stays NaN. Every other parameter is finite."""
    c = Case("f32", "f32", state, zero=True, seed=84)
    c.new_grads()
    bad = np.zeros(12345, dtype=bool)
    for i, x in {0: math.inf, 63: -math.inf, 64: math.nan, 4500: math.inf, 12344: math.nan}.items():
        c.grads[9][i] = x
        bad[i] = True
    c.opt.step(lr=1e-3)
    assert np.array_equal(np.isnan(f64(c.opt.params[0][9])), bad)
