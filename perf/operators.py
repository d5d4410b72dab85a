"""The optimizer step that follows a gradient synchronisation, as measured cases.

Three operators over many tensors at once: the global norm of the averaged
gradients with its clip coefficient, an AdamW step with 32-bit states, and an
AdamW step with 8-bit states. ``run`` computes them in their plain form, with
elementary torch operations on flat buffers, or (``own``) through the package.

With t the number of the step, per element:

    g'  = g * (grad_scale * coef)
    m   = b1 m + (1 - b1) g'
    v   = b2 v + (1 - b2) g' g'
    r   = sqrt(v)
    p   = p (1 - lr wd) - lr / (1 - b1^t) * m / (r / sqrt(1 - b2^t) + eps)

The 8-bit states hold m and r (v = r r). Each block of 64 consecutive elements
of a tensor has a power-of-two scale 2^(s - 127), s one byte (e8m0), the
smallest with max|x| <= 448 * scale; an element is an e4m3 code of x / scale,
rounded stochastically: down, or up when the fraction of a step that is left
plus u / 65536 reaches 1, with u of 16 bits from a hash of the optimizer's
seed, t and the element's index. r > 0 never becomes code 0. A code or scale is
returned as the value it stands for: torch's float8 tensors of those bytes.
"""
import math
import random

import torch

own = False

BETAS = (0.9, 0.999)
EPS = 1e-8
LR = 1e-4
WEIGHT_DECAY = 0.01
MAX_NORM = 1.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 64
M32 = 0xFFFFFFFF


# ---- the cases -------------------------------------------------------------------

def _linear():
    return [100, 10]


def _ragged():
    return [1, 3, 4097, 8193, 12345, 64, 20000, 5, 70000, 2, 777, 4096, 0, 16384, 33000]


def _resnet50():
    ps, c = [64 * 3 * 49, 64, 64], 64
    for si, (blocks, w) in enumerate([(3, 64), (4, 128), (6, 256), (3, 512)]):
        for b in range(blocks):
            ps += [w * c, w, w, w * w * 9, w, w, 4 * w * w, 4 * w, 4 * w]
            if b == 0:
                ps += [4 * w * c, 4 * w, 4 * w]
            c = 4 * w
    return ps + [1000 * 2048, 1000]


def _bert_large():
    h, f = 1024, 4096
    layer = [h * h, h] * 4 + [h, h, f * h, f, h * f, h, h, h]
    return [30522 * h, 512 * h, 2 * h, h, h] + layer * 24 + [h * h, h]


def _mlp():
    d, f = 2048, 8192
    return [f * d, f, d * f, d] * 24


SETS = {"linear10": _linear, "ragged": _ragged, "resnet50": _resnet50, "bert_large": _bert_large, "mlp": _mlp}


def _numels(case):
    if case["set"] in SETS:
        return SETS[case["set"]]()
    # "drawn": `elements` split over `tensors` with log-uniform weights
    rng = random.Random(case["split"])
    w = [math.exp(rng.uniform(0.0, 6.0)) for _ in range(case["tensors"])]
    return [max(1, int(case["elements"] * x / sum(w))) for x in w]


def _case(name, op, set_, p="f32", g="f32", state="f32", master=False, R=1, align=64, t=1000, loss_scale=1.0, **more):
    c = {"op": op, "set": set_, "p": p, "g": g, "state": state, "master": master, "R": R, "align": align, "t": t,
         "loss_scale": loss_scale, **more}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the smallest model of the pages (nn.Linear(10, 10), two replicas): what one step costs at least
        _case("adamw linear", "step", "linear10", R=2, t=0),
        # odd sizes and addresses, half-precision parameters with fp32 masters, a loss scale to take out
        _case("adamw ragged fp16", "step", "ragged", p="f16", g="f16", master=True, align=1, loss_scale=1024.0),
        # 161 tensors, most of them tiny; one set of states, eight replicas' parameters written
        _case("adamw resnet50 R8", "step", "resnet50", R=8),
        # a language model trained in fp32
        _case("adamw bert-large", "step", "bert_large"),
        # the same in mixed precision: bf16 parameters and gradients, fp32 masters
        _case("adamw bert-large bf16", "step", "bert_large", p="bf16", g="bf16", master=True),
        # 8-bit states: the smallest call
        _case("adamw8 linear", "step", "linear10", state="f8", t=0),
        # 8-bit states beside fp32 parameters, convolution shapes
        _case("adamw8 resnet50", "step", "resnet50", state="f8"),
        # 8-bit states, everything else in bf16: the least memory a step can do with
        _case("adamw8 bert-large bf16", "step", "bert_large", p="bf16", g="bf16", state="f8"),
        # the gradient norm of a tiny model: latency
        _case("norm linear", "norm", "linear10"),
        # the norm of a language model's fp32 gradients, as they lie after a synchronisation
        _case("norm bert-large", "norm", "bert_large"),
        # the norm of many bf16 gradients (the 24-layer MLP), packed without gaps
        _case("norm mlp bf16", "norm", "mlp", g="bf16", align=1),
        # a whole training step's end: norm, clip coefficient, 8-bit step
        _case("clip + adamw8 bert-large", "clip", "bert_large", state="f8"),
    ]


def draw(rng):
    op = rng.choice(["step", "step", "step", "norm", "clip"])
    g = rng.choice(["f32", "f32", "bf16", "f16"])
    p = rng.choice(["f32", g])
    state = rng.choice(["f32", "f8"])
    c = _case(None, op, "drawn", p=p, g=g, state=state, master=p != "f32" and rng.random() < 0.5,
              R=rng.choice([1, 1, 1, 2, 5, 8]), align=64 if state == "f8" and op != "norm" else rng.choice([1, 64]),
              t=rng.choice([0, 1, 10, 1000, 100000]), loss_scale=rng.choice([1.0, 256.0]))
    top = work(listed()[3])["bytes"]
    per = work({**c, "tensors": 1, "elements": 1 << 20, "split": 0})["bytes"] / (1 << 20)
    n = int(math.exp(rng.uniform(math.log(100), math.log(0.9 * min(top / per, 3e8)))))
    return {**c, "elements": n, "tensors": min(n, int(math.exp(rng.uniform(0, math.log(400))))),
            "split": rng.randrange(1 << 30)}


def work(case):
    ns = _numels(case)
    n, g = sum(ns), SIZE[case["g"]]
    if case["op"] == "norm":
        return {"bytes": n * g + 8, "flops": 2 * n}
    states = 2 * (2 * n + 2 * sum(-(-k // BLOCK) for k in ns)) if case["state"] == "f8" else 16 * n
    par = (8 + case["R"] * SIZE[case["p"]]) * n if case["master"] else (1 + case["R"]) * SIZE[case["p"]] * n
    # g' (1), m (3), v (4), r (1), p (6); clipping adds a pass over the gradients
    clip = case["op"] == "clip"
    return {"bytes": n * g * (2 if clip else 1) + states + par, "flops": (15 + 2 * clip) * n}


# ---- inputs ------------------------------------------------------------------------

def _offsets(ns, align):
    off, at = [], 0
    for n in ns:
        off.append(at)
        at += -(-n // align) * align
    return off, at


def prepare(case, seed):
    ns = _numels(case)
    off, total = _offsets(ns, case["align"])
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda: torch.randn(total, generator=gen, device="cuda")  # noqa: E731
    inside = None                      # the gaps between the tensors hold zeros
    if total != sum(ns):
        edge = torch.zeros(total + 1, dtype=torch.int32, device="cuda")
        one = torch.ones(len(ns), dtype=torch.int32, device="cuda")
        edge.index_put_((torch.tensor(off, device="cuda"),), one, accumulate=True)
        edge.index_put_((torch.tensor([o + n for o, n in zip(off, ns)], device="cuda"),), -one, accumulate=True)
        inside = torch.cumsum(edge[:-1], 0, dtype=torch.int32) > 0
        del edge
    put = lambda x: x if inside is None else x.mul_(inside)  # noqa: E731
    g = put(rnd().mul_(1e-3))
    rows = total // 10 // 1024         # embedding rows of tokens that the batch did not hold
    if rows:
        g[:rows * 1024].view(rows, 1024).mul_(torch.rand(rows, 1, generator=gen, device="cuda") > 0.3)
    s = {"case": case, "t": case["t"], "seed": seed % 1000003}
    s["g"] = g.mul_(case["loss_scale"]).to(DTYPES[case["g"]])
    del g
    if case["op"] != "norm":
        w = put(rnd().mul_(0.02))
        s["p"] = w.to(DTYPES[case["p"]]).expand(case["R"], total).contiguous()
        s["w"] = w if case["master"] else None
        if not case["master"]:
            del w
        if case["t"]:
            m = put(rnd().mul_(3e-4))
            r = put(rnd().abs_().mul_(4e-4).add_(6e-4))
        else:
            m, r = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
        if case["state"] == "f8":
            um, ur = _random16(s["seed"], case["t"], total)
            s["m"], s["ms"] = _encode(m, um, False)
            s["r"], s["rs"] = _encode(r, ur, True)
        else:
            s["m"], s["v"] = m, r.square_()
    if own:
        import ddp_bucketed_gradient_amd as D
        cut = lambda x: [x[o:o + n] for o, n in zip(off, ns)]  # noqa: E731
        grads = cut(s["g"])
        if case["op"] != "step":
            s["norm"] = D.GradNorm(grads)
        if case["op"] != "norm":
            if case["state"] == "f8":
                blocks = [-(-n // BLOCK) for n in ns]
                scl = lambda x: [x[o // BLOCK:o // BLOCK + b] for o, b in zip(off, blocks)]  # noqa: E731
                states = {"exp_avg": cut(s["m"]), "exp_avg_root": cut(s["r"]), "avg_scale": scl(s["ms"]),
                          "root_scale": scl(s["rs"])}
            else:
                states = {"exp_avg": cut(s["m"]), "exp_avg_sq": cut(s["v"])}
            s["opt"] = D.AdamW([cut(row) for row in s["p"]], grads, lr=LR, betas=BETAS, eps=EPS,
                               weight_decay=WEIGHT_DECAY, state=case["state"], master=cut(s["w"]) if case["master"] else None,
                               states=states, step=case["t"], seed=s["seed"])
    return s


# ---- one pass ------------------------------------------------------------------------

def run(s):
    case = s["case"]
    scale = 1.0 / case["loss_scale"]
    out = {}
    if own:
        clip = None
        if case["op"] != "step":
            clip = s["norm"]
            out["norm"] = clip.compute(max_norm=MAX_NORM, grad_scale=scale)
            out["coef"] = clip.coef
        if case["op"] != "norm":
            s["opt"].step(grad_scale=scale, clip=clip)
    else:
        coef = None
        if case["op"] != "step":
            out["norm"], out["coef"] = _norm(s["g"], scale)
            coef = out["coef"]
        if case["op"] != "norm":
            s["t"] += 1
            _step(s, scale, coef)
    if case["op"] != "norm":
        out["params"] = s["p"]
        if case["master"]:
            out["master"] = s["w"]
        out["exp_avg"] = s["m"]
        if case["state"] == "f8":
            out.update(exp_avg_root=s["r"], avg_scale=s["ms"], root_scale=s["rs"])
        else:
            out["exp_avg_sq"] = s["v"]
    return out


# ---- the plain form ------------------------------------------------------------------

def _norm(g, scale):
    norm = g.double().square_().sum().sqrt() * scale
    return norm.float(), torch.where(norm > MAX_NORM, MAX_NORM / norm, torch.ones_like(norm)).float()


def _step(s, scale, coef):
    t, f8 = s["t"], s["case"]["state"] == "f8"
    g = s["g"].float() * (scale if coef is None else coef * scale)
    m = _decode(s["m"], s["ms"]) if f8 else s["m"]
    v = _decode(s["r"], s["rs"]).square_() if f8 else s["v"]
    m = m * BETAS[0] + g * (1.0 - BETAS[0])
    v = v * BETAS[1] + (g * g) * (1.0 - BETAS[1])
    r = v.sqrt()
    w = s["w"] if s["w"] is not None else s["p"][0].float()
    step = LR / (1.0 - BETAS[0] ** t)
    w = w * (1.0 - LR * WEIGHT_DECAY) - (m / (r * (1.0 / math.sqrt(1.0 - BETAS[1] ** t)) + EPS)) * step
    s["p"].copy_(w)
    if s["w"] is not None:
        s["w"].copy_(w)
    if f8:
        um, ur = _random16(s["seed"], t, g.numel())
        code, sc = _encode(m, um, False)
        s["m"].copy_(code), s["ms"].copy_(sc)
        code, sc = _encode(r, ur, True)
        s["r"].copy_(code), s["rs"].copy_(sc)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def _decode(codes, scales):
    f = (scales.view(torch.uint8).int() << 23).view(torch.float32)
    return (codes.float().view(-1, BLOCK) * f[:, None]).view(-1)


def _encode(x, u16, root):
    """e4m3 codes and e8m0 scales of the blocks of x."""
    x = x.view(-1, BLOCK)
    fine = torch.isfinite(x)
    top = torch.where(fine, x.abs(), 0.0).amax(1).view(torch.int32)
    s = ((top >> 23) + ((top & 0x7FFFFF) > 0x600000).int() - 8).clamp_(min=1)
    y = x.abs() * ((254 - s) << 23).view(torch.float32)[:, None]
    low = (y < 2.0 ** -6).float() * 2.0 ** -6            # below it all steps are 2^-9
    z = (((y + low).view(torch.int32) + (u16.view(-1, BLOCK) << 4)) & ~0xFFFFF).view(torch.float32) - low
    if root:
        z = torch.where(y > 0, z.clamp(min=2.0 ** -9), z)
    z = torch.where(fine, torch.copysign(z, x), math.nan)
    return z.to(torch.float8_e4m3fn).view(-1), s.to(torch.uint8).view(torch.float8_e8m0fnu)


def _key(seed, t):
    m = (1 << 64) - 1
    k = (seed + t * 0xA3B1956C7E4D2F89) & m
    k ^= k >> 32
    k = k * 0xD6C7F2A94B1E8653 & m
    k ^= k >> 29
    k = k * 0x9E6B3F85C2D4A717 & m
    k ^= k >> 32
    return k & M32, k >> 32


def _random16(seed, t, total):
    """The 16 random bits of each element for m and for r: one hash per four elements, a short one per element."""
    k0, k1 = _key(seed, t)
    i = torch.arange(total // 4, device="cuda", dtype=torch.int64)
    h = ((i & M32) * 0x9C8E5A6D + (i >> 32) * 0x7F4A3C15 + k0) & M32
    h = ((h ^ (h >> 15)) * 0x85D3B2A7) & M32
    h = ((h ^ (h >> 13) ^ k1) * 0xC5A7E36B) & M32
    h = h ^ (h >> 16)
    x = (h[:, None] + torch.arange(4, device="cuda", dtype=torch.int64) * 0x6D2B4E95) & M32
    x = ((x ^ (x >> 16)) * 0xB5297A4D) & M32
    x = (x ^ (x >> 15)).view(-1)
    return (x >> 16).int(), (x & 0xFFFF).int()


# ---- the definition in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    g = s["g"].double()
    out, coef = {}, 1.0
    if case["op"] != "step":
        norm = float(torch.linalg.vector_norm(g)) / case["loss_scale"]
        coef = MAX_NORM / norm if norm > MAX_NORM else 1.0
        out["norm"], out["coef"] = norm, coef
        if case["op"] == "norm":
            return out
    g.mul_(coef / case["loss_scale"])
    t, (b1, b2), f8 = case["t"] + 1, BETAS, case["state"] == "f8"
    if f8:
        m, v = _values(s["m"], s["ms"]), _values(s["r"], s["rs"]) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = torch.lerp(g, m, b1)
    v = torch.lerp(g ** 2, v, b2)
    w = (s["w"] if case["master"] else s["p"][0]).double()
    w = w - LR * (WEIGHT_DECAY * w + (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + EPS))
    out["params"] = w.expand(case["R"], -1)
    if case["master"]:
        out["master"] = w
    if f8:
        um, ur = _random16(s["seed"], t, w.numel())
        out["exp_avg"], out["avg_scale"] = _nearby(m, um, False)
        out["exp_avg_root"], out["root_scale"] = _nearby(v.sqrt(), ur, True)
    else:
        out["exp_avg"], out["exp_avg_sq"] = m, v
    return out


def _values(codes, scales):
    """Codes and scales by the formats' definitions: sign, 4 exponent and 3 fraction bits; 2^(s - 127)."""
    c = torch.arange(256, dtype=torch.float64, device="cuda")
    e, f = torch.div(c % 128, 8, rounding_mode="floor"), c % 8
    value = torch.where(e > 0, (8 + f) * 2.0 ** (e - 10), f * 2.0 ** -9) * torch.where(c < 128, 1.0, -1.0)
    x = value[codes.view(torch.uint8).int()]
    return (x.view(-1, BLOCK) * 2.0 ** (scales.view(torch.uint8).double() - 127)[:, None]).view(-1)


def _nearby(x, u16, root):
    """The code values and scale values of x, block by block."""
    a = x.abs().view(-1, BLOCK)
    f, e = torch.frexp(a.amax(1))                      # max = f 2^e, f in [1/2, 1)
    scale = 2.0 ** (e - 9 + (f > 0.875)).clamp(min=-126).double()
    y = a / scale[:, None]
    q = 2.0 ** ((torch.frexp(y)[1] - 1).clamp(min=-6) - 3).double()
    z = torch.floor(y / q + u16.view(-1, BLOCK) / 65536.0) * q
    if root:
        z = torch.where(y > 0, z.clamp(min=2.0 ** -9), z)
    return torch.copysign(z.view(-1), x), scale
