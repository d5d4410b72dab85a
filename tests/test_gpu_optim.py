"""The gradient norm and the AdamW step on the GPU against the 64-bit oracle:
element types, odd sizes and addresses, replicas, special values, clipping,
skipped steps, graphs, streams, a tensor beyond 32-bit offsets, and a run of
synchronisation, norm and step together.

Tolerances are the oracle's bounds of an fp32 computation with one rounding per
operation (first order; 1 % covers the higher orders, which are U^2), and half a
step where a parameter is stored in 16 bits.
"""
import math

import numpy as np
import pytest
import torch

import ddp_bucketed_gradient_amd as D
from gpu_util import require_gpu, say
from oracle import optim as OO

pytestmark = pytest.mark.gpu

NUMELS = [1, 3, 64, 65, 0, 255, 4096, 4097, 2, 12345, 8192, 7]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}    # half a step below the normal range
GUARD = 0x5A


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.synchronize()


def f64(t):
    return t.detach().cpu().double().numpy()


def raw(t):
    return t.detach().cpu().reshape(-1).view(torch.uint8).numpy().copy()


class Storage:
    """Tensors packed one after the other (``gap`` elements between them) from
    ``lead`` elements into one buffer of guard bytes."""

    def __init__(self, numels, dtype, lead=0, gap=0):
        size = torch.empty(0, dtype=dtype).element_size()
        total = lead + sum(n + gap for n in numels) + 64
        self.bytes = torch.full((total * size,), GUARD, dtype=torch.uint8, device="cuda")
        self.inside = np.zeros(total * size, dtype=bool)
        self.tensors, at = [], lead
        for n in numels:
            self.tensors.append(self.bytes[at * size:(at + n) * size].view(dtype))
            self.inside[at * size:(at + n) * size] = True
            at += n + gap

    def assert_guards(self, what):
        b = self.bytes.cpu().numpy()
        assert (b[~self.inside] == GUARD).all(), f"{what}: wrote outside its tensors"


class Case:
    """Parameters, gradients and state in guarded storages, and their AdamW."""

    def __init__(self, p="f32", g="f32", state="f32", master=False, R=1, lead=0, gap=0, numels=NUMELS, seed=1,
                 zero=False, random_seed=0, **opt):
        self.numels, self.p, self.g, self.f8, self.R = numels, p, g, state == "f8", R
        self.stores = {}
        new = lambda name, ns, dt: self.stores.setdefault(name, Storage(ns, dt, lead, gap)).tensors  # noqa: E731
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gen = gen
        rnd = lambda n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
        rows = [new(f"params{r}", numels, TYPES[p]) for r in range(R)]
        self.grads = new("grads", numels, TYPES[g])
        w = [rnd(n) * 0.02 for n in numels]
        for row in rows:
            for t, x in zip(row, w):
                t.copy_(x)
        ms = new("master", numels, torch.float32) if master else None
        if master:
            for t, x in zip(ms, w):
                t.copy_(x)
        blocks = [-(-n // 64) for n in numels]
        kinds = {"exp_avg": torch.float8_e4m3fn, "exp_avg_root": torch.float8_e4m3fn,
                 "avg_scale": torch.float8_e8m0fnu, "root_scale": torch.float8_e8m0fnu} if self.f8 else \
            {"exp_avg": torch.float32, "exp_avg_sq": torch.float32}
        states = {k: new(k, blocks if k.endswith("scale") else numels, dt) for k, dt in kinds.items()}
        for k, ts in states.items():
            for t in ts:
                n = t.numel()
                if zero:
                    t.view(torch.uint8).zero_()
                elif k.endswith("scale"):             # around 1e-3 / 448
                    t.view(torch.uint8).copy_(torch.randint(106, 112, (n,), generator=gen, device="cuda"))
                elif self.f8:                         # every code but NaN; roots are not negative
                    c = torch.randint(0, 127, (n,), generator=gen, device="cuda", dtype=torch.int32)
                    if k == "exp_avg":
                        c += 128 * torch.randint(0, 2, (n,), generator=gen, device="cuda", dtype=torch.int32)
                    t.view(torch.uint8).copy_(c)
                else:
                    t.copy_(rnd(n) * 1e-3 if k == "exp_avg" else (rnd(n) * 1e-3) ** 2)
        self.wd = opt.setdefault("weight_decay", 0.01)
        self.lr_scale = opt.get("lr_scale")
        self.seed, self.t = random_seed, opt.get("step", 0)
        self.eps, self.betas = opt.get("eps", 1e-8), opt.get("betas", (0.9, 0.999))
        self.opt = D.AdamW(rows if R > 1 else rows[0], self.grads, state=state, master=ms, states=states,
                           seed=random_seed, **opt)

    def new_grads(self, scale=1e-3):
        for t in self.grads:
            t.copy_(torch.randn(t.numel(), generator=self.gen, device="cuda") * scale)

    def host(self):
        """Everything as fp64 host arrays, by variable."""
        o = self.opt
        src = o.master if o.master is not None else o.params[0]
        out = {"w": [f64(t) for t in src], "g": [f64(t) for t in self.grads]}
        if self.f8:
            dec = lambda c, s: OO.decode(raw(c), raw(s)) if c.numel() else np.zeros(0)  # noqa: E731
            out["m"] = [dec(c, s) for c, s in zip(o.exp_avg, o.avg_scale)]
            out["v"] = [dec(c, s) ** 2 for c, s in zip(o.exp_avg_root, o.root_scale)]
        else:
            out["m"], out["v"] = [f64(t) for t in o.exp_avg], [f64(t) for t in o.exp_avg_sq]
        return out

    def check_step(self, before, lr, gscale, what=""):
        """The state now against one step from ``before``."""
        torch.cuda.synchronize()
        self.t += 1
        every = lambda x, v, d: d if x is None else x if isinstance(x, float) else x[v]  # noqa: E731
        index = OO.bases(self.numels)
        for v, n in enumerate(self.numels):
            if n == 0:
                continue
            tag = f"{what} step {self.t} variable {v} ({n})"
            (w, m, vv, r), (bw, bm, bv, br) = OO.adamw(
                before["w"][v], before["g"][v], before["m"][v], before["v"][v], t=self.t,
                lr=lr * every(self.lr_scale, v, 1.0), beta1=self.betas[0], beta2=self.betas[1], eps=self.eps,
                weight_decay=every(self.wd, v, 0.0), gscale=gscale)
            o = self.opt
            p0 = o.params[0][v]
            if o.master is not None:
                close(f64(o.master[v]), w, bw, tag + " master")
                want = o.master[v].cpu().to(TYPES[self.p])
                assert np.array_equal(raw(p0), raw(want)), tag + " parameter is not the rounded master"
            else:
                half = 0.0 if self.p == "f32" else torch.finfo(TYPES[self.p]).eps / 2
                close(f64(p0), w, bw + half * (np.abs(w) + bw) + (TINY[self.p] if half else 0.0), tag + " param")
            for row in o.params[1:]:
                assert np.array_equal(raw(row[v]), raw(p0)), tag + " replica"
            if self.f8:
                um, ur = OO.random16(self.seed, self.t, index[v] + np.arange(n, dtype=np.uint64))
                check_codes(m, bm, um, False, raw(o.exp_avg[v]), raw(o.avg_scale[v]), tag + " m")
                check_codes(r, br, ur, True, raw(o.exp_avg_root[v]), raw(o.root_scale[v]), tag + " r")
            else:
                close(f64(o.exp_avg[v]), m, bm, tag + " m")
                close(f64(o.exp_avg_sq[v]), vv, bv, tag + " v")
        for k, s in self.stores.items():
            s.assert_guards(f"{what} {k}")


def close(got, want, bound, what):
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN elsewhere"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what + ": infinities"
    off = np.abs(got[fine] - want[fine]) - 1.01 * np.broadcast_to(bound, want.shape)[fine] - 2.0 ** -148
    assert (off <= 0).all(), f"{what}: off by {off.max():.3g} more than the bound, at {int(off.argmax())}"


def check_codes(x, bound, u16, root, codes, scales, what):
    """Codes and scales against those of the values from x - bound to x +
    bound: rounding with fixed random bits does not decrease anywhere."""
    fine = np.isfinite(x)
    vals = OO.CODES[codes]
    assert np.array_equal(np.isnan(vals), ~fine), what + ": NaN codes"
    x, bound = np.where(fine, x, 0.0), np.where(fine, 1.01 * bound, 0.0) + 2.0 ** -148
    a = np.abs(x)
    lo, hi = OO.scales_of(np.where(a > 2 * bound, a - bound, 0.0)), OO.scales_of(np.where(a > 0, a + bound, 0.0))
    s = scales.astype(np.int64)
    assert ((lo <= s) & (s <= hi)).all(), what + ": scales"
    unit = np.repeat(np.ldexp(1.0, s - 127), 64)[:x.size]
    # |x| / scale + 2^-6 rounds once more below 2^-6: 2^-30 at most there
    slack = bound + unit * 2.0 ** -30

    def at(y):
        low, up, pos = OO.encode_levels(np.maximum(y, 0.0), s, u16, root)
        return np.where(pos >= 1, up, low)
    got = np.abs(np.where(fine, vals, 0.0))
    assert ((at(a - slack) <= got) & (got <= at(a + slack))).all(), what + ": codes"
    sure = fine & (a > slack) & (got > 0)
    assert (np.signbit(vals[sure]) == np.signbit(x[sure])).all(), what + ": signs"
    if root:
        assert (got[fine & (x > slack)] > 0).all(), what + ": a root became 0"


# ---- AdamW ------------------------------------------------------------------------------

KINDS = [("f32", g, False) for g in TYPES] + [(p, g, m) for p in ("bf16", "f16") for g in TYPES for m in (False, True)]


@pytest.mark.parametrize("state", ["f32", "f8"])
@pytest.mark.parametrize("p,g,master", KINDS)
def test_three_steps_match_the_oracle(p, g, master, state):
    say(f"adamw p={p} g={g} master={master} state={state}")
    c = Case(p, g, state, master, seed=3, step=17)
    for lr, gs in ((1e-3, 1.0), (2e-2, 0.5), (0.0, 3.0)):
        c.new_grads()
        before = c.host()
        c.opt.step(lr=lr, grad_scale=gs)
        c.check_step(before, lr, gs, f"{p}/{g}/{master}/{state}")
    assert c.opt.steps_done == 20


@pytest.mark.parametrize("state", ["f32", "f8"])
@pytest.mark.parametrize("p,master", [("f32", False), ("bf16", True), ("f16", False)])
@pytest.mark.parametrize("lead,gap", [(1, 0), (3, 1), (2, 5)])
def test_odd_addresses(p, master, state, lead, gap):
    """Tensors packed without regard to alignment: element-aligned vectors, code
    words at odd bytes, nothing written between them."""
    c = Case(p, "bf16" if p == "f32" else p, state, master, R=2, lead=lead, gap=gap, seed=lead)
    c.new_grads()
    before = c.host()
    c.opt.step(lr=1e-2)
    c.check_step(before, 1e-2, 1.0, f"odd {p} {state}")


@pytest.mark.parametrize("state", ["f32", "f8"])
@pytest.mark.parametrize("R", [2, 5, 64])
def test_replicas_receive_row_zero(R, state):
    c = Case("f32", "f32", state, R=R, numels=[5, 4100, 64], seed=R)
    for row in c.opt.params[1:]:
        for t in row:
            t.fill_(7.0)                             # not read
    c.new_grads()
    before = c.host()
    c.opt.step(lr=1e-2)
    c.check_step(before, 1e-2, 1.0, f"R={R}")


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_first_steps_from_zeros(state):
    c = Case("f32", "f32", state, zero=True, seed=5)
    for _ in range(3):
        c.new_grads()
        before = c.host()
        c.opt.step(lr=1e-3)
        c.check_step(before, 1e-3, 1.0, "zeros")


def test_states_made_by_the_class_start_at_zero():
    p = [torch.ones(n, device="cuda") for n in (5, 0, 130)]
    g = [torch.full((n,), 0.5, device="cuda") for n in (5, 0, 130)]
    for state in ("f32", "f8"):
        q = [t.clone() for t in p]
        opt = D.AdamW(q, g, lr=0.125, weight_decay=0.0, state=state)
        assert opt.steps_done == 0
        opt.step()                                   # the first step: lr * sign(g)
        assert opt.steps_done == 1
        for t in q:                                  # the update's relative bound: 5 + 13 roundings, eps / |g|
            assert (t - 0.875).abs().max().item() <= 0.125 * (18 * OO.U + 2e-8) + 3 * OO.U if t.numel() else True
        assert opt.exp_avg[2].shape == (130,) and opt.exp_avg[2].data_ptr() % 256 == 0


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_options_by_variable(state):
    n = len(NUMELS)
    c = Case("f32", "f32", state, seed=9, weight_decay=[0.1 * (v % 3) for v in range(n)],
             lr_scale=[0.0 if v == 7 else 0.5 + v for v in range(n)], betas=(0.0, 0.5), eps=1e-3)
    for _ in range(2):
        c.new_grads()
        before = c.host()
        c.opt.step(lr=1e-2)
        c.check_step(before, 1e-2, 1.0, "options")


@pytest.mark.parametrize("state", ["f32", "f8"])
@pytest.mark.parametrize("p", ["f32", "bf16"])
def test_special_gradients(p, state):
    """Infinities, NaN, zeros, subnormals and huge values touch their own
    elements only: the oracle's values in every other place."""
    c = Case(p, "f32", state, seed=11, zero=True)
    c.new_grads()
    big = c.grads[9]                                  # 12345 elements
    for i, x in {0: math.inf, 63: -math.inf, 64: math.nan, 200: 0.0, 201: -0.0, 202: 1e-40, 203: -1e-45, 300: 1e18,
                 12344: math.nan}.items():
        big[i] = x
    big[4096:4160] = 0.0                              # a block of zeros
    big[4160:4224] = math.nan                         # a block without a finite value
    big[4224:4288] = 1e-22                            # squares underflow to zero
    before = c.host()
    c.opt.step(lr=1e-3)
    # squares below the fp32 range round to multiples of 2^-149, which the relative bounds leave out:
    # compare those elements apart
    tiny = np.abs(before["g"][9]) < 1e-18
    got = f64(c.opt.params[0][9])
    torch.cuda.synchronize()
    assert np.isfinite(got[np.isfinite(before["g"][9])]).all()
    for i in np.flatnonzero(~np.isfinite(before["g"][9])):
        assert not np.isfinite(got[i]) or abs(got[i]) < 1
    keep = [k for k in range(12345) if not tiny[k] and np.isfinite(before["g"][9][k])]
    (w, m, vv, r), (bw, *_) = OO.adamw(before["w"][9], before["g"][9], before["m"][9], before["v"][9], t=1, lr=1e-3,
                                       beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, gscale=1.0)
    half = 0.0 if p == "f32" else 2.0 ** -8
    close(got[keep], w[keep], bw[keep] + half * np.abs(w[keep]) + (half > 0) * 2.0 ** -134, "special")
    if state == "f8":
        codes, scales = raw(c.opt.exp_avg[9]), raw(c.opt.avg_scale[9])
        bad = ~np.isfinite(before["g"][9])
        assert np.isnan(OO.CODES[codes[bad]]).all() and not np.isnan(OO.CODES[codes[~bad]]).any()
        assert scales[64] == 1 and scales[65] == 1    # blocks of zeros, of NaN only
        assert (codes[4096:4160] & 127 == 0).all()
    else:
        bad = ~np.isfinite(before["g"][9])
        assert not np.isfinite(f64(c.opt.exp_avg[9])[bad]).any()
        assert np.isfinite(f64(c.opt.exp_avg[9])[~bad]).all()


@pytest.mark.parametrize("g", ["f32", "f16"])
def test_codes_beside_special_gradients(g):
    """In the waves that hold infinities, NaN and values whose 2^64 v leaves fp32,
    every other element gets the codes and scales it would get alone."""
    c = Case("f32", g, "f8", seed=13, step=3)
    c.new_grads()
    big = c.grads[9]
    for i, x in {0: math.inf, 63: -math.inf, 64: math.nan, 200: 0.0, 201: -0.0, 300: 1e18 if g == "f32" else 6e4,
                 1024: math.nan, 5000: -math.inf, 12344: math.nan}.items():
        big[i] = x
    c.opt.exp_avg[10].view(torch.uint8)[5] = 0x7F       # a state that is NaN already, its root is not
    big[8192:8256] = math.inf                          # a block without a finite value
    before = c.host()
    c.opt.step(lr=1e-3)
    torch.cuda.synchronize()
    for v in (9, 10):
        n = c.numels[v]
        (w, m, vv, r), (bw, bm, bv, br) = OO.adamw(before["w"][v], before["g"][v], before["m"][v], before["v"][v], t=4,
                                                   lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
                                                   gscale=1.0)
        um, ur = OO.random16(0, 4, OO.bases(c.numels)[v] + np.arange(n, dtype=np.uint64))
        check_codes(m, bm, um, False, raw(c.opt.exp_avg[v]), raw(c.opt.avg_scale[v]), f"m {v}")
        check_codes(r, br, ur, True, raw(c.opt.exp_avg_root[v]), raw(c.opt.root_scale[v]), f"r {v}")
        fine = np.isfinite(w)
        close(f64(c.opt.params[0][v])[fine], w[fine], bw[fine], f"param {v}")
        assert not np.isfinite(f64(c.opt.params[0][v])[~fine]).any()


def test_same_bits_every_time():
    outs = []
    for _ in range(2):
        c = Case("bf16", "bf16", "f8", master=True, seed=21)
        c.new_grads()
        n = D.GradNorm(c.grads)
        n.compute(max_norm=0.01)
        c.opt.step(lr=1e-2, clip=n)
        torch.cuda.synchronize()
        outs.append([raw(n.norm), raw(n.coef)] + [s.bytes.cpu().numpy() for s in c.stores.values()])
    for a, b in zip(*outs):
        assert np.array_equal(a, b)


def test_tensor_beyond_32_bit_offsets():
    """2^32 + 193 elements in bf16 with 8-bit states: offsets past 32 bits in
    elements and bytes, blocks and random bits past 2^32."""
    n = (1 << 32) + 193
    say("adamw8 with 2^32 + 193 elements")
    p = torch.empty(n, dtype=torch.bfloat16, device="cuda").fill_(0.5)
    g = torch.empty(n, dtype=torch.bfloat16, device="cuda").fill_(0.25)
    opt = D.AdamW([p], [g], lr=1e-2, weight_decay=0.0, state="f8", seed=77)
    where = [0, 4096 * 5, (1 << 31) - 100, (1 << 32) - 100, n - 193]
    span = 193
    for k, a in enumerate(where):
        p[a:a + span] = torch.linspace(-1, 1, span, device="cuda") * (k + 1) * 0.01
        g[a:a + span] = torch.linspace(1e-3, 2e-3, span, device="cuda") * (k + 1)
    old = [(f64(p[a:a + span]), f64(g[a:a + span])) for a in where]
    norm = D.GradNorm([g])
    assert norm.compute().item() == pytest.approx(0.25 * math.sqrt(n), rel=1e-6)   # the spans weigh < 1e-6 of it
    opt.step()
    torch.cuda.synchronize()
    for a, (w0, g0) in zip(where, old):
        (w, m, v, r), (bw, bm, bv, br) = OO.adamw(w0, g0, 0.0 * w0, 0.0 * w0, t=1, lr=1e-2, beta1=0.9, beta2=0.999,
                                                  eps=1e-8, weight_decay=0.0, gscale=1.0)
        close(f64(p[a:a + span]), w, bw + 2.0 ** -8 * np.abs(w), f"at {a}")
        um, ur = OO.random16(77, 1, np.uint64(a) + np.arange(span, dtype=np.uint64))
        lo, hi = -(-a // 64), (a + span) // 64       # whole blocks inside the span
        if a + span == n:
            hi = -(-n // 64)
        for x, b, u, root, codes, scales in ((m, bm, um, False, opt.exp_avg[0], opt.avg_scale[0]),
                                             (r, br, ur, True, opt.exp_avg_root[0], opt.root_scale[0])):
            e = min(hi * 64, n)
            cut = slice(lo * 64 - a, e - a)
            check_codes(x[cut], b[cut], u[cut], root, raw(codes[lo * 64:e]), raw(scales[lo:hi]), f"codes at {a}")
    rest = p[1 << 20:1 << 21]
    assert (rest == rest[0]).all().item() and abs(rest[0].item() - 0.49) <= 0.49 * 2.0 ** -8


@pytest.mark.parametrize("seed", range(40))
def test_random_configurations(seed):
    """Types, sizes, addresses, replicas, options, steps and clipping drawn at
    random; two steps each."""
    rng = np.random.default_rng(1000 + seed)
    pick = lambda *xs: xs[int(rng.integers(len(xs)))]  # noqa: E731
    p = pick("f32", "bf16", "f16")
    P = int(rng.integers(1, 12))
    numels = [int(x) for x in np.exp(rng.uniform(0, math.log(pick(70, 3000, 30000)), P))]
    numels[int(rng.integers(P))] = pick(0, 1, 64, 256, 1024, 2048, 4096, 8191)
    betas = pick((0.9, 0.999), (0.0, 0.99), (0.5, 0.0), (0.95, 0.9999))
    opt = dict(weight_decay=[float(x) for x in rng.uniform(0, 0.2, P)], betas=betas, eps=pick(1e-8, 1e-6, 1e-15),
               random_seed=int(rng.integers(1 << 62)), step=int(pick(0, 1, 37, 10 ** 6)))
    if rng.random() < 0.5:
        opt["lr_scale"] = [float(x) for x in rng.uniform(0, 2, P)]
    g, state, master = pick("f32", "bf16", "f16"), pick("f32", "f8"), p != "f32" and rng.random() < 0.5
    R, lead, gap = pick(1, 1, 2, 5), pick(0, 0, 1, 2, 7), pick(0, 0, 1, 3)
    say(f"random {seed}: p={p} g={g} {state} master={master} R={R} lead={lead} gap={gap} {numels} {opt}")
    c = Case(p, g, state, master, R=R, lead=lead, gap=gap, numels=numels, seed=seed, **opt)
    n = D.GradNorm(c.grads) if rng.random() < 0.5 else None
    for _ in range(2):
        c.new_grads(scale=pick(1e-4, 1e-2, 1.0))
        lr, gs = float(10 ** rng.uniform(-5, -1)), float(pick(1.0, 1.0 / 512, -3.0))
        before = c.host()
        factor = gs
        if n is not None:
            n.compute(max_norm=0.1, grad_scale=gs, skip_nonfinite=True)
            want = OO.norm(before["g"], gs)
            assert abs(n.norm.item() - want) <= 2 * OO.U * want
            factor = gs * n.coef.item()
        c.opt.step(lr=lr, grad_scale=gs, clip=n)
        c.check_step(before, lr, factor, f"random {seed}")


# ---- norm -------------------------------------------------------------------------------

def _grads(numels, types, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * scale).to(TYPES[types[v % len(types)]])
            for v, n in enumerate(numels)]


@pytest.mark.parametrize("types", [["f32"], ["bf16"], ["f16"], ["f32", "bf16", "f16"]])
@pytest.mark.parametrize("numels", [[], [0], [1], [3, 0, 5], NUMELS, [4096 * 1024 + 4097] * 2])
def test_norm_matches_the_oracle(numels, types):
    """fp64 sums of n non-negative terms, at most n roundings of 2^-53 each
    (half of that for the root), then one to fp32."""
    say(f"norm {types} {numels}")
    g = _grads(numels, types, 5)
    n = D.GradNorm(g)
    for gs, mx in ((1.0, math.inf), (-0.25, 0.5)):
        got = n.compute(max_norm=mx, grad_scale=gs).item()
        want = float(torch.stack([t.double().square().sum() for t in g]).sum().sqrt()) * abs(gs) \
            if sum(numels) > 100000 else OO.norm([f64(t) for t in g], gs)
        tol = OO.U + (sum(numels) + 4) * 2.0 ** -53
        assert abs(got - want) <= tol * want
        assert abs(n.coef.item() - OO.clip_coef(want, mx)) <= (OO.U + 2 * tol) * OO.clip_coef(want, mx)
        assert n.skipped.item() == 0


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("lead,gap", [(1, 0), (3, 1), (5, 7)])
def test_norm_at_odd_addresses(t, lead, gap):
    """Guard bytes around the tensors (0x5A5A...: large or small numbers, never
    0) would show in the sum."""
    s = Storage(NUMELS, TYPES[t], lead, gap)
    for x, y in zip(s.tensors, _grads(NUMELS, [t], lead)):
        x.copy_(y)
    n = D.GradNorm(s.tensors)
    want = OO.norm([f64(x) for x in s.tensors])
    assert abs(n.compute().item() - want) <= (OO.U + sum(NUMELS) * 2.0 ** -53) * want


def test_norm_of_values_whose_squares_leave_fp32():
    n = D.GradNorm([torch.full((10000,), 1e30, device="cuda"), torch.full((3,), 1e-30, device="cuda")])
    assert n.compute().item() == pytest.approx(1e32, rel=2e-7)
    m = D.GradNorm([torch.full((10000,), 1e-30, device="cuda")])
    assert m.compute().item() == pytest.approx(1e-28, rel=2e-7)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("state", ["f32", "f8"])
def test_a_step_is_skipped_on_a_norm_that_is_not_finite(bad, state):
    c = Case("f32", "f32", state, seed=31)
    c.new_grads()
    good = [t.clone() for t in c.grads]
    c.grads[9][777] = bad
    n = D.GradNorm(c.grads)
    before = {k: s.bytes.cpu().numpy() for k, s in c.stores.items()}
    norm = n.compute(max_norm=1.0, skip_nonfinite=True)
    c.opt.step(lr=1e-2, clip=n)
    torch.cuda.synchronize()
    assert not math.isfinite(norm.item()) and n.skipped.item() == 1 and c.opt.steps_done == 0
    for k, s in c.stores.items():
        assert np.array_equal(before[k], s.bytes.cpu().numpy()), k
    for t, x in zip(c.grads, good):                   # the next one counts as the first
        t.copy_(x)
    old = c.host()
    n.compute(max_norm=1.0, skip_nonfinite=True)
    c.opt.step(lr=1e-2, clip=n)
    assert n.skipped.item() == 0
    c.check_step(old, 1e-2, 1.0, "after a skip")
    assert c.opt.steps_done == 1


def test_clip_scales_the_gradients():
    c = Case("f32", "bf16", "f32", seed=33)
    n = D.GradNorm(c.grads)
    for mx in (0.01, 100.0):
        c.new_grads(scale=0.1)
        before = c.host()
        n.compute(max_norm=mx, grad_scale=0.5)
        c.opt.step(lr=1e-2, grad_scale=0.5, clip=n)
        want = OO.clip_coef(OO.norm(before["g"], 0.5), mx)
        assert (want < 1) == (mx < 1)
        # the coefficient is rounded to fp32 before the factor is formed: within the gradient's 4 roundings + 1
        c.check_step(before, 1e-2, 0.5 * float(n.coef.item()), f"clip {mx}")


# ---- graphs and streams --------------------------------------------------------------------

@pytest.mark.parametrize("state", ["f32", "f8"])
def test_captured_norm_and_step_replay_like_eager_ones(state):
    """A captured norm and step, replayed with the program's own work and
    synchronizations between: the same bits as an eager twin, the count of steps
    and a rate in device memory moving along."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        a, b = (Case("f32", "f32", state, seed=41, stream=stream) for _ in range(2))
        na, nb = (D.GradNorm(c.grads, stream=stream) for c in (a, b))
        lr = torch.full((1,), 1e-2, device="cuda")
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        na.compute(max_norm=0.05, skip_nonfinite=True)
        a.opt.step(lr=lr, clip=na)
        for call in (lambda: a.opt.steps_done, lambda: setattr(a.opt, "steps_done", 3)):
            with pytest.raises(D.DdpbError) as e:
                call()
            assert e.value.code == D.E_STATE
    with torch.cuda.stream(stream):
        for rep in range(5):
            lr.fill_(1e-2 / (rep + 1))
            for c in (a, b):
                c.gen.manual_seed(1000 + rep)
                c.new_grads(scale=0.1 if rep % 2 else 1e-4)
                if rep == 2:
                    c.grads[5][3] = math.nan             # this one is skipped
            g.replay()
            nb.compute(max_norm=0.05, skip_nonfinite=True)
            b.opt.step(lr=lr, clip=nb)
            stream.synchronize()
            torch.randn(1000, device="cuda").sum().item()
            assert np.array_equal(raw(na.norm), raw(nb.norm))
            for k in a.stores:
                assert np.array_equal(a.stores[k].bytes.cpu().numpy(), b.stores[k].bytes.cpu().numpy()), (rep, k)
    assert a.opt.steps_done == b.opt.steps_done == 4


def test_bind_is_refused_during_capture():
    p, g = [torch.ones(10, device="cuda")], [torch.ones(10, device="cuda")]
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        x.add_(1)
        with pytest.raises(D.DdpbError) as e:
            D.GradNorm(g, stream=stream)
        assert e.value.code == D.E_STATE
    graph.replay()
    torch.cuda.synchronize()
    assert x.item() == 1 and p[0].sum().item() == 10


def test_work_runs_on_the_bound_stream():
    """A step bound to a side stream waits for that stream's work and for
    nothing else."""
    side = torch.cuda.Stream()
    c = Case("f32", "f32", "f32", seed=51, stream=side)
    other = torch.randn(c.grads[9].numel(), device="cuda")
    torch.cuda.synchronize()
    x = torch.randn(4096, 4096, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(20):
            x = x @ x * 1e-3                              # keeps the stream busy
        c.new_grads()
        c.grads[9].copy_(other)
    c.opt.step(lr=1e-2)                                   # enqueued from the default stream
    side.synchronize()
    # the step has run on these gradients: from the same start, a twin's one eager step
    twin = Case("f32", "f32", "f32", seed=51)
    twin.new_grads()
    twin.grads[9].copy_(other)
    torch.cuda.synchronize()
    before = twin.host()
    twin.opt.step(lr=1e-2)
    twin.check_step(before, 1e-2, 1.0, "twin")
    for k in c.stores:
        assert np.array_equal(c.stores[k].bytes.cpu().numpy(), twin.stores[k].bytes.cpu().numpy()), k


def test_two_handles_on_two_streams():
    """Norm and step of two models at once, each on its own stream: what each
    gives alone."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = []
    for k, st in enumerate(streams):
        with torch.cuda.stream(st):
            c = Case("f32", "bf16", "f8" if k else "f32", seed=70 + k, stream=st)
            both.append((c, D.GradNorm(c.grads, stream=st)))
    twins = [(c, D.GradNorm(c.grads)) for c in (Case("f32", "bf16", "f8" if k else "f32", seed=70 + k)
                                                for k in range(2))]
    torch.cuda.synchronize()
    for _ in range(5):
        for (c, n), st in zip(both, streams):
            with torch.cuda.stream(st):
                c.new_grads()
                n.compute(max_norm=0.02)
                c.opt.step(lr=1e-2, clip=n)
    torch.cuda.synchronize()
    for c, n in twins:
        for _ in range(5):
            c.new_grads()
            n.compute(max_norm=0.02)
            c.opt.step(lr=1e-2, clip=n)
            torch.cuda.synchronize()
    for (c, _), (d, _) in zip(both, twins):
        for k in c.stores:
            assert np.array_equal(c.stores[k].bytes.cpu().numpy(), d.stores[k].bytes.cpu().numpy()), k


def test_masters_are_made_from_what_the_caller_enqueued():
    side = torch.cuda.Stream()
    p = [torch.zeros(100000, dtype=torch.bfloat16, device="cuda")]
    g = [torch.zeros(100000, device="cuda")]
    x = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        x = x @ x * 1e-3                                  # keeps the current stream busy
    p[0].fill_(0.75)
    opt = D.AdamW(p, g, master=True, stream=side, lr=0.0)
    opt.step()
    side.synchronize()
    assert (opt.master[0] == 0.75).all().item() and (p[0] == 0.75).all().item()


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_a_new_handle_goes_on_bit_for_bit(state):
    a, b = (Case("bf16", "f32", state, master=True, seed=65, step=9) for _ in range(2))
    for rep in range(4):
        for c in (a, b):
            c.new_grads()
        a.opt.step(lr=1e-2)
        b.opt.step(lr=1e-2)
        old = b.opt
        b.opt = D.AdamW(old.params[0], old.grads, state=state, master=old.master, states=old.states,
                        step=old.steps_done, weight_decay=0.01)
        old.close()
    torch.cuda.synchronize()
    assert a.opt.steps_done == b.opt.steps_done == 13
    for k in a.stores:
        assert np.array_equal(a.stores[k].bytes.cpu().numpy(), b.stores[k].bytes.cpu().numpy()), k


def test_a_modules_parameters():
    """nn.Module.parameters(), gradients of autograd, a NumPy rate; one step of
    torch's arithmetic in fp64."""
    torch.manual_seed(3)
    m = torch.nn.Sequential(torch.nn.Linear(33, 70), torch.nn.GELU(), torch.nn.Linear(70, 5)).cuda()
    m(torch.randn(16, 33, device="cuda")).square().mean().backward()
    old = [f64(p) for p in m.parameters()]
    opt = D.AdamW(m.parameters(), [p.grad for p in m.parameters()], weight_decay=0.1)
    opt.step(lr=np.float32(0.25))
    for p, w0 in zip(m.parameters(), old):
        (w, *_), (bw, *_) = OO.adamw(w0, f64(p.grad), 0 * w0, 0 * w0, t=1, lr=0.25, beta1=0.9, beta2=0.999, eps=1e-8,
                                     weight_decay=0.1, gscale=1.0)
        close(f64(p), w, bw, "module")
    opt = D.AdamW(list(m.bfloat16().parameters()), [p.grad.float() for p in m.parameters()], master=True)
    assert not any(w.requires_grad for w in opt.master)


def test_set_step():
    c = Case("f32", "f32", "f8", seed=61, step=5)
    c.opt.steps_done = 100000
    c.t = 100000
    c.new_grads()
    before = c.host()
    c.opt.step(lr=1e-2)
    c.check_step(before, 1e-2, 1.0, "set_step")
    assert c.opt.steps_done == 100001


# ---- refusals of the Python front end --------------------------------------------------------

def test_python_refusals():
    f = lambda n=10, dt=torch.float32: torch.ones(n, dtype=dt, device="cuda")  # noqa: E731
    bad = [
        lambda: D.AdamW([f()], [f(11)]), lambda: D.AdamW([f(), f()], [f()]),
        lambda: D.AdamW([f(10, torch.float64)], [f()]), lambda: D.AdamW([f()], [f(10, torch.int32)]),
        lambda: D.AdamW([f(), f(10, torch.bfloat16)], [f(), f()]), lambda: D.AdamW([f().cpu()], [f()]),
        lambda: D.AdamW([f(20)[::2]], [f()]), lambda: D.AdamW([f()], [f(20)[::2]]),
        lambda: D.AdamW([f()], [f()], state="f16"), lambda: D.AdamW([f()], [f()], states={"exp_avg": [f()]}),
        lambda: D.AdamW([f()], [f()], states={"exp_avg": [f()], "exp_avg_sq": [f(9)]}),
        lambda: D.AdamW([f(10, torch.bfloat16)], [f()], master=[f(10, torch.bfloat16)]),
        lambda: D.AdamW([f()], [f()], weight_decay=[0.1, 0.1]), lambda: D.GradNorm([f().cpu()]),
        lambda: D.AdamW([f(), f()], [f(), None]), lambda: D.AdamW([f()], [None]), lambda: D.GradNorm([f(), None]),
        lambda: D.AdamW([f()], [f().cpu()]), lambda: D.AdamW([f(), None], [f(), f()]),
        lambda: D.GradNorm([f(10, torch.int32)]), lambda: D.GradNorm([f(20)[::2]]),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {k} was not refused")
    with pytest.raises(D.DdpbError):                       # a tied parameter listed twice
        t = f()
        D.AdamW([t, t], [f(), f()])
    with pytest.raises(D.DdpbError):
        D.AdamW([f()], [f()], master=True)                 # fp32 parameters need no master
    opt = D.AdamW([f()], [f()])
    side = torch.cuda.Stream()
    for kw in (dict(lr="1e-3"), dict(lr=torch.ones(1)), dict(lr=f(2)), dict(lr=f(1, torch.bfloat16)),
               dict(clip=D.GradNorm([f()], stream=side))):
        with pytest.raises(ValueError):
            opt.step(**kw)
    opt.close()
    opt.close()


def test_nothing_to_update():
    opt = D.AdamW([], [])
    n = D.GradNorm([])
    assert n.compute(max_norm=1.0).item() == 0.0
    opt.step(clip=n)
    assert opt.steps_done == 1
    opt = D.AdamW([torch.empty(0, device="cuda")], [torch.empty(0, device="cuda")], state="f8")
    opt.step()
    assert opt.steps_done == 1


# ---- a training step as it is used -------------------------------------------------------------

def test_groups_share_one_norm_behind_a_sync():
    """Matrices with 8-bit states and decay, vectors with 32-bit states and none:
    two handles on one reducer's gradients, one coefficient for both."""
    shapes = [(33, 31), (33,), (64, 70), (64,), (4097, 2)]
    R, rng = 2, np.random.default_rng(8)
    red = D.Reducer(shapes, R, 4 * 3000)
    grads = [[torch.from_numpy(rng.normal(size=s).astype(np.float32)).cuda() for s in shapes] for _ in range(R)]
    red.bind(grads)
    params = [torch.from_numpy(rng.normal(size=s).astype(np.float32) * 0.02).cuda() for s in shapes]
    big, small = [0, 2, 4], [1, 3]
    norm = red.grad_norm()
    opts = [D.AdamW([params[v] for v in vs], [grads[0][v] for v in vs], weight_decay=wd, state=st, reducer=red)
            for vs, wd, st in ((big, 0.1, "f8"), (small, 0.0, "f32"))]
    old = [f64(p) for p in params]
    red.sync()
    norm.compute(max_norm=0.5)
    for o in opts:
        o.step(lr=1e-2, clip=norm)
    torch.cuda.synchronize()
    g = [f64(x) for x in grads[0]]
    coef = OO.clip_coef(OO.norm(g), 0.5)
    assert coef < 1 and abs(norm.coef.item() - coef) <= 4 * OO.U * coef
    for v in range(len(shapes)):
        (w, *_), (bw, *_) = OO.adamw(old[v], g[v], 0 * g[v], 0 * g[v], t=1, lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8,
                                     weight_decay=0.1 if v in big else 0.0, gscale=norm.coef.item())
        close(f64(params[v]), w, bw, f"variable {v}")
    red.close()


@pytest.mark.parametrize("state", ["f32", "f8"])
@pytest.mark.parametrize("view", [False, True])
def test_synchronise_clip_and_step(view, state):
    """Three training steps of R replicas: hooks, buckets, averaged gradients,
    norm, clip, AdamW into every replica; wrong moments are refused."""
    shapes = [(5,), (33, 31), (4100,), (0,), (64, 2), (3,), (9000,)]
    numels = [math.prod(s) for s in shapes]
    R, rng = 3, np.random.default_rng(5)
    red = D.Reducer(shapes, R, 4 * 5000)
    if view:
        grads = red.bind_bucket_views()
    else:
        grads = [[torch.empty(s, device="cuda") for s in shapes] for _ in range(R)]
        red.bind(grads)
    init = [rng.normal(size=s).astype(np.float32) * 0.02 for s in shapes]
    params = [[torch.from_numpy(x.copy()).cuda() for x in init] for _ in range(R)]
    norm = red.grad_norm()
    opt = red.adamw(params, lr=1e-2, weight_decay=0.1, state=state, seed=9)
    m, v = [np.zeros(n) for n in numels], [np.zeros(n) for n in numels]
    for t in range(1, 4):
        local = [[rng.normal(size=s).astype(np.float32) * 0.1 for s in shapes] for _ in range(R)]
        for r in range(R):
            for x, y in zip(grads[r], local[r]):
                x.copy_(torch.from_numpy(y))
        red.mark_ready(len(shapes) - 1)
        for call in (lambda: norm.compute(max_norm=1.0), opt.step):
            with pytest.raises(D.DdpbError) as e:
                call()
            assert e.value.code == D.E_STATE
        old = [f64(x).ravel() for x in params[0]]
        for k in reversed(range(len(shapes) - 1)):
            red.mark_ready(k)
        red.finalize()
        norm.compute(max_norm=1.0)
        opt.step(clip=norm)
        torch.cuda.synchronize()
        mean = [f64(x).ravel() for x in grads[0]]
        for k in range(len(shapes)):
            np.testing.assert_allclose(mean[k], np.mean([y[k] for y in local], axis=0, dtype=np.float64).ravel(),
                                       rtol=0, atol=4 * OO.U * 0.6)        # 3 roundings of sums below 0.6
        coef = OO.clip_coef(OO.norm(mean), 1.0)
        assert coef < 1 and abs(norm.coef.item() - coef) <= 4 * OO.U * coef
        for k, n in enumerate(numels):
            if state == "f8" and n:
                if t > 1:
                    m[k], v[k] = prev[k]
            (w, mm, vv, _), (bw, bm, bv, _) = OO.adamw(old[k], mean[k], m[k], v[k], t=t, lr=1e-2, beta1=0.9,
                                                       beta2=0.999, eps=1e-8, weight_decay=0.1,
                                                       gscale=norm.coef.item())
            if state == "f32":
                close(f64(opt.exp_avg[k]), mm, bm, f"m {k}")
                close(f64(opt.exp_avg_sq[k]), vv, bv, f"v {k}")
                m[k], v[k] = f64(opt.exp_avg[k]), f64(opt.exp_avg_sq[k])
            for r in range(R):
                close(f64(params[r][k]).ravel(), w, bw, f"step {t} replica {r} variable {k}")
        if state == "f8":
            prev = [(OO.decode(raw(opt.exp_avg[k]), raw(opt.avg_scale[k])),
                     OO.decode(raw(opt.exp_avg_root[k]), raw(opt.root_scale[k])) ** 2) if n else (np.zeros(0),) * 2
                    for k, n in enumerate(numels)]
    if view:
        red.bind_bucket_views()
    else:
        red.bind(grads)
    for call in (lambda: norm.compute(max_norm=1.0), opt.step):     # the binding they were made for is gone
        with pytest.raises(D.DdpbError) as e:
            call()
        assert e.value.code == D.E_STATE
    red.grad_norm().compute()
    red.close()
    for call in (lambda: norm.compute(max_norm=1.0), opt.step):
        with pytest.raises(D.DdpbError) as e:
            call()
        assert e.value.code == D.E_STATE
    torch.cuda.synchronize()
