"""The operators beside the matrix products of a data-parallel model, as measured cases.

Layer norm (with a residual and dropout in front of it), dropout from a
counter-based generator and the embedding lookup: forward passes, and backward
passes whose parameter gradients go where the reducer finds them. ``run``
computes them in their plain form, with elementary torch operations in fp32, or
(``own``) through the package.

Dropout   keeps element i where u_i >= T, T = round(65536 p), and divides what
          it keeps by 1 - T / 65536. u_i is the 16-bit half i % 2 of word
          i % 8 / 2 of Philox4x32 with 7 rounds (Salmon et al. 2011) of the
          counter (i / 8, offset), two 64-bit numbers, under the seed as key; i
          counts the elements row by row.
Norm      z = residual + drop(x), n = (z - mean z) s, s = 1 / sqrt(var z + eps),
          y = n w + b.  Gradients, with g = dy w:  dz = s (g - mean g -
          n mean(g n)) + what else reaches z;  dx = drop(dz);  dw = sum dy n,
          db = sum dy over the rows.
Lookup    y_i = scale table[t_i] + residual_i;  dtable[v] = scale * sum of the
          dy_i with t_i = v. A token outside of the table gives zeros.
"""
import functools
import math

import torch

own = False

EPS = 1e-5
SCALE = 0.5
OFFSET = (3 << 32) + 5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
M32 = 0xFFFFFFFF


# ---- the cases -------------------------------------------------------------------

def _norm(name, op, rows, cols, t, w="f32", g="f32", residual=False, p=0.0, more=False, add=False, pad=0):
    """w, g: types of the weights and of their gradients; residual, p: what stands in front of the norm; more: another
    gradient reaches z; add: the weights' gradients are added to; pad: elements between the rows of the inputs."""
    c = {"op": op, "rows": rows, "cols": cols, "t": t, "w": w, "g": g, "residual": residual, "p": p, "more": more,
         "add": add, "pad": pad}
    return {"name": name, **c} if name else c


def _drop(name, rows, cols, t, p=0.1, residual=False, pad=0):
    c = {"op": "dropout", "rows": rows, "cols": cols, "t": t, "p": p, "residual": residual, "pad": pad}
    return {"name": name, **c} if name else c


def _look(name, op, n, vocab, cols, t, w="f32", residual=False, add=False, padded=0.0, ignored=0.0):
    """t: the type of y or dy; w: of the table or its gradient; padded: the share of tokens that are 0 (the end of short
    sequences); ignored: the share of tokens that are -1."""
    c = {"op": op, "n": n, "vocab": vocab, "cols": cols, "t": t, "w": w, "residual": residual, "add": add,
         "padded": padded, "ignored": ignored}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token of a served model: what a call costs at least
        _norm("norm one token", "norm", 1, 1024, "bf16"),
        # the end of a sublayer of BERT-large, 32 sequences of 512 tokens: residual and dropout in front
        _norm("norm bert-large", "norm", 16384, 1024, "bf16", residual=True, p=0.1),
        # its backward pass: the gradients of both branches and of the weights, as the reducer takes them
        _norm("norm gradient bert-large", "norm_grad", 16384, 1024, "bf16", residual=True, p=0.1),
        # odd sizes, rows cut out of a wider tensor, half-precision weights, a local step that is added
        _norm("norm gradient ragged fp16", "norm_grad", 3001, 771, "f16", w="f16", g="f16", more=True, add=True, pad=5),
        # the inner width of the MLP over 8192 tokens in fp32, a norm of a block's input: two gradients meet
        _norm("norm gradient wide fp32", "norm_grad", 8192, 8192, "f32", more=True),
        # the batch of the smallest model: latency
        _drop("dropout linear", 20, 10, "f32", p=0.5),
        # the MLP's activations over 8192 tokens
        _drop("dropout mlp", 8192, 8192, "bf16"),
        # half precision, odd sizes, with a residual
        _drop("dropout ragged fp16", 2049, 1533, "f16", p=0.3, residual=True, pad=3),
        # BERT-large's words, 32 sequences of 512 tokens, from the fp32 parameter
        _look("lookup bert-large", "lookup", 16384, 30522, 1024, "bf16"),
        # their gradient, the whole table of it, a variable of the first bucket that is full last
        _look("lookup gradient bert-large", "lookup_grad", 16384, 30522, 1024, "bf16"),
        # a local step over many short sequences of BERT-base: one token holds 40 % of the places, others are left out
        _look("lookup gradient padded", "lookup_grad", 131072, 30522, 768, "bf16", add=True, padded=0.4, ignored=0.1),
        # the front of BERT-base, 16 sequences of 512: words and positions, norm, dropout, forward and backward
        _look("front bert-base", "front", 8192, 30522, 768, "f32"),
    ]


def draw(rng):
    top = max(work(c)["bytes"] for c in listed())
    size = lambda a, b: int(math.exp(rng.uniform(math.log(a), math.log(b + 1))))  # noqa: E731
    while True:
        op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "dropout", "dropout", "lookup", "lookup_grad",
                         "lookup_grad", "front"])
        t = rng.choice(["f32", "bf16", "f16"])
        w = rng.choice(["f32", "f32", t])
        if op in ("norm", "norm_grad"):
            drop = rng.choice([0.0, 0.0, 0.1, 0.25])
            c = _norm(None, op, size(1, 65536), size(1, 16384), t, w, rng.choice(["f32", "f32", t]),
                      drop > 0 or rng.random() < 0.3, drop, rng.random() < 0.3, rng.random() < 0.3,
                      rng.choice([0, 0, 1, 8]))
        elif op == "dropout":
            c = _drop(None, size(1, 65536), size(1, 32768), t, rng.choice([0.0, 0.1, 0.5, 0.9]), rng.random() < 0.5,
                      rng.choice([0, 0, 1, 8]))
        else:
            padded = rng.choice([0.0, 0.0, 0.3, 0.8])
            c = _look(None, op, size(1, 262144), size(2, 262144), size(1, 4096), t, w, rng.random() < 0.3,
                      rng.random() < 0.4, padded, rng.choice([0.0, 0.05]))
        if op == "front":
            c["residual"], c["add"], c["padded"], c["ignored"] = False, False, 0.0, 0.0
        if work(c)["bytes"] <= top and c.get("vocab", 0) * c["cols"] <= 1 << 28:
            return c


@functools.lru_cache(None)
def _distinct(n, vocab):
    """Tokens of a table that n draws hit, on average: rank k has the share log(1 + 1 / k) / log(vocab + 1)."""
    top = math.log(vocab + 1)
    return max(1, round(sum(1.0 - (1.0 - math.log1p(1.0 / k) / top) ** n for k in range(1, vocab + 1))))


def work(case):
    c, s = case, SIZE[case["t"]]
    if case["op"] in ("norm", "norm_grad", "dropout"):
        n = c["rows"] * c["cols"]
        if c["op"] == "dropout":
            return {"bytes": n * s * (2 + c["residual"]), "flops": n * (2 + c["residual"])}
        fused = c["residual"] or c["p"] > 0
        if c["op"] == "norm":
            # mean (1), squares (3), normalise (2), weights (2)
            return {"bytes": n * s * (2 + c["residual"] + fused) + 8 * c["rows"] + 2 * c["cols"] * SIZE[c["w"]],
                    "flops": n * (8 + c["residual"] + 2 * (c["p"] > 0))}
        # n (2), g (1), two sums (3), dz (4), weights' sums (3)
        return {"bytes": n * s * (3 + c["more"] + (c["p"] > 0)) + 8 * c["rows"]
                + c["cols"] * (SIZE[c["w"]] + 2 * SIZE[c["g"]] * (1 + c["add"])),
                "flops": n * (13 + c["more"] + 2 * (c["p"] > 0))}
    cols, table = c["cols"], SIZE[c["w"]]
    here = round(c["n"] * (1.0 - c["ignored"]))
    hit = _distinct(max(1, round(here * (1.0 - c["padded"]))), c["vocab"]) + (c["padded"] > 0)
    look = {"bytes": 8 * c["n"] + hit * cols * table + c["n"] * cols * s * (1 + c["residual"]),
            "flops": c["n"] * cols * (1 + c["residual"])}
    grad = {"bytes": 8 * c["n"] + here * cols * s + cols * table * (2 * hit if c["add"] else c["vocab"]),
            "flops": (c["n"] + hit) * cols}
    if c["op"] == "lookup":
        return look
    if c["op"] == "lookup_grad":
        return grad
    # tokens, words, positions, weights and dy in; y and the gradients out
    n, pos = c["n"] * cols, _positions(c)
    return {"bytes": 16 * c["n"] + cols * table * (hit + 2 * pos + c["vocab"] + 4) + 2 * n * s, "flops": n * 30}


def _positions(case):
    return min(512, case["n"])


# ---- inputs ------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    t, op, cols = DTYPES[case["t"]], case["op"], case["cols"]
    s = {"case": case, "seed": seed * 0x9E3779B97F4A7C15 & (1 << 64) - 1}
    if op in ("norm", "norm_grad", "dropout"):
        rows = case["rows"]

        def cut(x):                            # a view of rows that lie `pad` elements apart
            wide = torch.zeros(rows, cols + case["pad"], dtype=t, device="cuda")
            wide[:, :cols].copy_(x)
            return wide[:, :cols]
        # activations with a few strong channels and an offset, as trained networks have them
        chan = 1.0 + 4.0 * (torch.rand(cols, generator=gen, device="cuda") > 0.98)
        s["x"] = cut(rnd(rows, cols) * chan + 0.3)
        if case["residual"]:
            s["residual"] = cut(rnd(rows, cols) * chan)
        if op != "dropout":
            wt, gt = DTYPES[case["w"]], DTYPES[case["g"]]
            s["w"] = (1.0 + 0.1 * rnd(cols)).to(wt)
            s["b"] = (0.1 * rnd(cols)).to(wt)
        if op == "norm_grad":
            z = s["h"] = s["x"]                # what the forward pass left
            del s["x"]
            s.pop("residual", None)
            z = z.float()
            m = z.mean(1, keepdim=True)
            s["stats"] = torch.cat([m, 1.0 / torch.sqrt((z - m).square_().mean(1, keepdim=True) + EPS)], 1)
            del z
            s["dy"] = cut(rnd(rows, cols) * 0.01)
            if case["more"]:
                s["dh"] = cut(rnd(rows, cols) * 0.01)
            s["dw"], s["db"] = (0.01 * rnd(cols)).to(gt), (0.01 * rnd(cols)).to(gt)
    else:
        vocab, w = case["vocab"], DTYPES[case["w"]]
        u = torch.rand(case["n"], generator=gen, device="cuda", dtype=torch.float64)
        rank = torch.exp(u * math.log(vocab + 1)).long().clamp_(1, vocab) - 1
        step = next(k for k in (7919, 7927, 7933, 7937) if math.gcd(k, vocab) == 1)
        tokens = (rank * step + 17) % vocab
        for share, token in ((case["padded"], 0), (case["ignored"], -1)):
            if share:                          # sequences of 128 end early, all lengths alike around the mean
                low = max(0.0, 1.0 - 2 * share)
                length = low + 2 * (1.0 - share - low) * torch.rand(-(-case["n"] // 128), 1, generator=gen, device="cuda")
                end = torch.arange(128, device="cuda") / 128 >= length
                tokens = torch.where(end.view(-1)[:case["n"]], token, tokens)
        s["tokens"] = tokens
        if op in ("lookup", "front"):
            s["table"] = (0.02 * rnd(vocab, cols)).to(w)
        if op == "lookup" and case["residual"]:
            s["residual"] = (0.02 * rnd(case["n"], cols)).to(t)
        if op in ("lookup_grad", "front"):
            s["dy"] = (0.01 * rnd(case["n"], cols)).to(t)
            s["dtable"] = (0.01 * rnd(vocab, cols)).to(w)
        if op == "front":
            pos = _positions(case)
            s["places"] = torch.arange(case["n"], device="cuda") % pos
            s["where"] = (0.02 * rnd(pos, cols)).to(w)
            s["dwhere"] = torch.zeros_like(s["where"])
            s["w"], s["b"] = (1.0 + 0.1 * rnd(cols)).to(w), (0.1 * rnd(cols)).to(w)
            s["dw"], s["db"] = torch.zeros_like(s["w"]), torch.zeros_like(s["b"])
    if own:
        import ddp_bucketed_gradient_amd as D
        s["D"] = D
        p = 0.1 if op == "front" else case.get("p", 0.0)
        s["drop"] = D.Drop(p, s["seed"], OFFSET) if p > 0 or op == "dropout" else None
    return s


# ---- one pass ------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    D, c = s["D"], s["case"]
    if c["op"] == "norm":
        n = D.layer_norm(s["x"], s["w"], s["b"], EPS, residual=s.get("residual"), drop=s["drop"])
        return {"y": n.y, "stats": n.stats, **({"h": n.h} if n.h is not s["x"] else {})}
    if c["op"] == "norm_grad":
        g = D.layer_norm_backward(s["dy"], s["h"], s["stats"], s["w"], s["dw"], s["db"], grad_h=s.get("dh"),
                                  drop=s["drop"], accumulate=c["add"])
        return {"dh": g.dh, **({"dx": g.dx} if c["p"] > 0 else {}), "dw": s["dw"], "db": s["db"]}
    if c["op"] == "dropout":
        return D.dropout(s["x"], s["drop"], residual=s.get("residual"))
    if c["op"] == "lookup":
        return D.embedding(s["tokens"], s["table"], SCALE, residual=s.get("residual"), dtype=DTYPES[c["t"]])
    if c["op"] == "lookup_grad":
        D.embedding_backward(s["dy"], s["tokens"], s["dtable"], SCALE, accumulate=c["add"])
        return s["dtable"]
    # in fp32 throughout, as mixed precision keeps its norms: the parameters' gradients are fp32
    f = torch.float32
    words = D.embedding(s["tokens"], s["table"], SCALE, dtype=f)
    n = D.layer_norm(D.embedding(s["places"], s["where"], residual=words, dtype=f), s["w"], s["b"], EPS)
    y = D.dropout(n.y, s["drop"]).to(DTYPES[c["t"]])
    dy = D.dropout_backward(s["dy"].float(), s["drop"])
    dh = D.layer_norm_backward(dy, n.h, n.stats, s["w"], s["dw"], s["db"]).dh
    D.embedding_backward(dh, s["tokens"], s["dtable"], SCALE)
    D.embedding_backward(dh, s["places"], s["dwhere"])
    return {"y": y, "dtable": s["dtable"], "dwhere": s["dwhere"], "dw": s["dw"], "db": s["db"]}


# ---- the plain form ------------------------------------------------------------------

def _run_plain(s):
    c = s["case"]
    t = DTYPES[c["t"]]
    if c["op"] == "norm":
        z = s["x"].float()
        if c["p"] > 0:
            z = _dropped(z, s["seed"], c["p"])
        if c["residual"]:
            z = z + s["residual"].float()
        y, stats = _normed(z, s["w"], s["b"])
        return {"y": y.to(t), "stats": stats, **({"h": z.to(t)} if c["residual"] or c["p"] > 0 else {})}
    if c["op"] == "norm_grad":
        dh, dw, db = _norm_grads(s["dy"].float(), s["h"].float(), s["stats"], s["w"])
        if c["more"]:
            dh = dh + s["dh"].float()
        for to, d in ((s["dw"], dw), (s["db"], db)):
            to.copy_(to.float() + d if c["add"] else d)
        return {"dh": dh.to(t), **({"dx": _dropped(dh, s["seed"], c["p"]).to(t)} if c["p"] > 0 else {}),
                "dw": s["dw"], "db": s["db"]}
    if c["op"] == "dropout":
        y = _dropped(s["x"].float(), s["seed"], c["p"])
        return (y + s["residual"].float() if c["residual"] else y).to(t)
    if c["op"] == "lookup":
        y = _looked(s["tokens"], s["table"], SCALE)
        return (y + s["residual"].float() if c["residual"] else y).to(t)
    if c["op"] == "lookup_grad":
        d = _look_grad(s["dy"].float(), s["tokens"], c["vocab"], SCALE)
        s["dtable"].copy_(s["dtable"].float() + d if c["add"] else d)
        return s["dtable"]
    z = _looked(s["tokens"], s["table"], SCALE) + _looked(s["places"], s["where"], 1.0)
    n, stats = _normed(z, s["w"], s["b"])
    y = _dropped(n, s["seed"], 0.1)
    dh, dw, db = _norm_grads(_dropped(s["dy"].float(), s["seed"], 0.1), z, stats, s["w"])
    s["dtable"].copy_(_look_grad(dh, s["tokens"], c["vocab"], SCALE))
    s["dwhere"].copy_(_look_grad(dh, s["places"], _positions(c), 1.0))
    s["dw"].copy_(dw), s["db"].copy_(db)
    return {"y": y.to(t), "dtable": s["dtable"], "dwhere": s["dwhere"], "dw": s["dw"], "db": s["db"]}


def _dropped(x, seed, p):
    limit = round(65536 * p)
    if limit == 0:
        return x
    keep = _random16(seed, OFFSET, x.numel()).view(x.shape) >= limit
    return torch.where(keep, x * (65536 / (65536 - limit)), 0.0)


def _random16(seed, offset, n):
    """16 random bits for each of n elements."""
    i = torch.arange(-(-n // 8), device="cuda", dtype=torch.int64)
    x = [i & M32, i >> 32, torch.full_like(i, offset & M32), torch.full_like(i, offset >> 32)]
    k0, k1 = seed & M32, seed >> 32
    for _ in range(7):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57       # the low 64 bits, of which the sign is one
        x = [(b >> 32 & M32) ^ x[1] ^ k0, b & M32, (a >> 32 & M32) ^ x[3] ^ k1, a & M32]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return torch.stack([h for w in x for h in (w & 0xFFFF, w >> 16)], 1).view(-1)[:n]


def _normed(z, w, b):
    mean = z.mean(1, keepdim=True)
    c = z - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    return c * rstd * w.float() + b.float(), torch.cat([mean, rstd], 1)


def _norm_grads(dy, z, stats, w):
    n = (z - stats[:, :1]) * stats[:, 1:]
    g = dy * w.float()
    dz = (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True)) * stats[:, 1:]
    return dz, (dy * n).sum(0), dy.sum(0)


def _looked(tokens, table, scale):
    inside = (tokens >= 0) & (tokens < table.shape[0])
    return torch.where(inside[:, None], table[torch.where(inside, tokens, 0)].float() * scale, 0.0)


def _look_grad(dy, tokens, vocab, scale):
    inside = (tokens >= 0) & (tokens < vocab)
    d = torch.zeros(vocab, dy.shape[1], device="cuda")
    return d.index_add_(0, tokens[inside], dy[inside]) * scale


# ---- the definition in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c, f = case, torch.float64
    if c["op"] == "norm":
        z = s["x"].to(f) * _mask(s, c["p"])
        if c["residual"]:
            z += s["residual"]
        var, mean = torch.var_mean(z, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(s["b"].to(f), (z - mean[:, None]) * rstd[:, None], s["w"].to(f))
        return {"y": y, "stats": torch.stack([mean, rstd], 1), **({"h": z} if c["residual"] or c["p"] > 0 else {})}
    if c["op"] == "norm_grad":
        dh, dw, db = _exact_norm_grads(s["dy"].to(f), s["h"].to(f), s["stats"].to(f), s["w"].to(f))
        if c["more"]:
            dh += s["dh"]
        if c["add"]:
            dw, db = dw + s["dw"], db + s["db"]
        return {"dh": dh, **({"dx": dh * _mask(s, c["p"])} if c["p"] > 0 else {}), "dw": dw, "db": db}
    if c["op"] == "dropout":
        y = s["x"].to(f) * _mask(s, c["p"])
        return y + s["residual"] if c["residual"] else y
    if c["op"] == "lookup":
        y = SCALE * _rows_of(s["tokens"], s["table"])
        return y + s["residual"] if c["residual"] else y
    if c["op"] == "lookup_grad":
        d = SCALE * _sums_of(s["dy"].to(f), s["tokens"], c["vocab"])
        return d + s["dtable"] if c["add"] else d
    z = SCALE * _rows_of(s["tokens"], s["table"]) + _rows_of(s["places"], s["where"])
    var, mean = torch.var_mean(z, 1, correction=0)
    stats = torch.stack([mean, (var + EPS) ** -0.5], 1)
    mask = _mask(s, 0.1, z.shape)
    n = (z - stats[:, :1]) * stats[:, 1:]
    dh, dw, db = _exact_norm_grads(s["dy"] * mask, z, stats, s["w"].to(f))
    return {"y": torch.addcmul(s["b"].to(f), n, s["w"].to(f)) * mask,
            "dtable": SCALE * _sums_of(dh, s["tokens"], c["vocab"]),
            "dwhere": _sums_of(dh, s["places"], _positions(c)), "dw": dw, "db": db}


def _exact_norm_grads(dy, z, stats, w):
    n = (z - stats[:, :1]) * stats[:, 1:]
    g = torch.mul(dy, w)
    mean_gn = torch.linalg.vecdot(g, n)[:, None] / z.shape[1]
    dz = stats[:, 1:] * (g - g.sum(1, keepdim=True) / z.shape[1] - mean_gn * n)
    return dz, torch.linalg.vecdot(dy, n, dim=0), dy.sum(0)


def _mask(s, p, shape=None):
    """What each element is multiplied by."""
    limit = math.floor(65536 * p + 0.5)
    shape = s["dy" if "dy" in s else "x"].shape if shape is None else shape
    if limit == 0:
        return torch.ones(shape, dtype=torch.float64, device="cuda")
    n = shape[0] * shape[1]
    g = torch.arange((n + 7) // 8, device="cuda", dtype=torch.int64)
    c0, c1 = g % 2 ** 32, g // 2 ** 32
    c2, c3 = torch.zeros_like(g) + OFFSET % 2 ** 32, torch.zeros_like(g) + OFFSET // 2 ** 32

    def product(x, m):                         # 32 by 32 bits in 16-bit halves: high and low word
        xl, xh, ml, mh = x % 65536, x // 65536, m % 65536, m // 65536
        low, mid = xl * ml, xl * mh
        mid2 = xh * ml + low // 65536 + mid % 65536
        return xh * mh + mid // 65536 + mid2 // 65536, (mid2 % 65536) * 65536 + low % 65536
    for r in range(7):
        h0, l0 = product(c0, 0xD2511F53)
        h1, l1 = product(c2, 0xCD9E8D57)
        k0 = (s["seed"] + r * 0x9E3779B9) % 2 ** 32
        k1 = (s["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
    m = torch.empty(g.numel(), 8, dtype=torch.float64, device="cuda")
    for j, word in enumerate((c0, c1, c2, c3)):
        m[:, 2 * j] = word % 65536 >= limit
        m[:, 2 * j + 1] = word // 65536 >= limit
    return m.view(-1)[:n].view(shape) / (1.0 - limit / 65536)


def _rows_of(tokens, table):
    padded = torch.cat([table, torch.zeros_like(table[:1])]).double()
    return padded.index_select(0, torch.where((tokens < 0) | (tokens >= table.shape[0]), table.shape[0], tokens))


def _sums_of(dy, tokens, vocab):
    """Sums of the rows of each token, from running sums over the rows in order of their tokens."""
    key = torch.where((tokens < 0) | (tokens >= vocab), vocab, tokens)
    order = torch.argsort(key)
    run = torch.cat([torch.zeros_like(dy[:1]), torch.cumsum(dy[order], 0)])
    ends = torch.bincount(key, minlength=vocab + 1)[:vocab].cumsum(0)
    return torch.diff(run[ends], dim=0, prepend=run[:1])
