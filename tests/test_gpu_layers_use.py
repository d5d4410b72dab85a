"""Layer norm, dropout and the embedding as a program uses them: a run of them
together against 64-bit autograd, through the reducer to the optimizer step, on
other streams, in graphs, and the front end's refusals."""
import numpy as np
import pytest
import torch

import ddp_bucketed_gradient_amd as D
from gpu_util import require_gpu, say
from oracle import layers as OL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.synchronize()


VOCAB, POS, H = 211, 24, 72
SHAPES = [(VOCAB, H), (POS, H), (H,), (H,), (H,), (H,)]      # words, positions, two norms


class Front:
    """words + positions -> norm -> dropout -> sublayer (here: a factor) ->
    norm of residual and dropout; forward and backward through the package."""

    def __init__(self, tokens, params, dy, seed=11, counter=None):
        self.tokens, self.params, self.dy = tokens, params, dy
        self.places = (torch.arange(tokens.numel(), device="cuda") % POS).view(tokens.shape)
        self.drops = [D.Drop(0.1, seed, i, counter) for i in range(2)]

    def forward(self):
        words, where, w1, b1, w2, b2 = self.params
        z = D.embedding(self.places, where, residual=D.embedding(self.tokens, words, 3.0, dtype=self.dy.dtype),
                        dtype=self.dy.dtype)
        self.n1 = D.layer_norm(z, w1, b1)
        self.y1 = D.dropout(self.n1.y, self.drops[0])
        self.n2 = D.layer_norm(self.y1 * 0.5, w2, b2, residual=self.y1, drop=self.drops[1])
        return self.n2.y

    def backward(self, grads, accumulate=False):
        words, where, w1, b1, w2, b2 = grads
        g = D.layer_norm_backward(self.dy, self.n2.h, self.n2.stats, self.params[4], w2, b2, drop=self.drops[1],
                                  accumulate=accumulate)
        d = D.dropout_backward(g.dh + g.dx * 0.5, self.drops[0])
        d = D.layer_norm_backward(d, self.n1.h, self.n1.stats, self.params[2], w1, b1, accumulate=accumulate).dh
        D.embedding_backward(d, self.tokens, words, 3.0, accumulate)
        D.embedding_backward(d, self.places, where, accumulate=accumulate)


def inputs(seed, dtype=torch.float32, n=(5, 40)):
    g = torch.Generator().manual_seed(seed)
    tokens = torch.randint(-1, VOCAB, n, generator=g)
    tokens[:, -7:] = 0
    params = [torch.randn(s, generator=g) * (0.1 if len(s) == 2 else 0.3) + (len(s) == 1) for s in SHAPES]
    dy = torch.randn(*n, H, generator=g).to(dtype)
    return tokens.cuda(), [p.cuda() for p in params], dy.cuda()


def autograd(tokens, params, dy, seed=11, offset=0):
    """The same in 64 bits on the CPU."""
    ps = [p.double().cpu().requires_grad_() for p in params]
    t, n = tokens.cpu(), tokens.numel()
    masks = [torch.from_numpy(OL.factors((n, H), 0.1, seed, offset + i)).view(*t.shape, H) for i in range(2)]
    words, where, w1, b1, w2, b2 = ps
    z = words[t.clamp(min=0)] * 3.0 * (t >= 0)[..., None] + where[torch.arange(n).view(t.shape) % POS]

    def norm(z, w, b):
        d = z - z.mean(-1, keepdim=True)
        return d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5) * w + b
    y1 = norm(z, w1, b1) * masks[0]
    y2 = norm(y1 + y1 * 0.5 * masks[1], w2, b2)
    y2.backward(dy.double().cpu())
    return y2.detach(), [p.grad for p in ps]


def close(got, want, tol):
    """Against the largest value: the chain is a dozen operations deep, each a few
    roundings off, and sums over 200 places."""
    err = (got.double().cpu() - want).abs().max() / want.abs().max()
    assert err < tol, err


# fp32: some 12 operations of at most ~40 roundings of 2^-24 each; bf16: about 10
# activations rounded once each, 2^-8 of their value, with factors of rstd |w| < 4
@pytest.mark.parametrize("dtype, tol", [(torch.float32, 12 * 40 * 2.0 ** -24), (torch.bfloat16, 10 * 4 * 2.0 ** -8)])
def test_a_run_of_them_against_autograd(dtype, tol):
    tokens, params, dy = inputs(1, dtype)
    f = Front(tokens, params, dy)
    grads = [torch.full(s, float("nan"), device="cuda") for s in SHAPES]
    y = f.forward()
    f.backward(grads)
    want, wants = autograd(tokens, params, dy)
    close(y, want, tol)
    for a, b in zip(grads, wants):
        close(a, b, tol)
    before = [g.clone() for g in grads]
    f.backward(grads, accumulate=True)
    for a, b in zip(grads, before):
        assert torch.allclose(a, 2 * b, rtol=2.0 ** -22, atol=0)


def replicas(R, seed=0):
    _, params, _ = inputs(seed)
    return [Front(*(lambda i: (i[0], params, i[2]))(inputs(seed + 1 + r)), seed=100 + r) for r in range(R)], params


def through_reducer(red, fronts, accumulate=False):
    for f in fronts:
        f.forward()
    n2, n1 = [f.n2 for f in fronts], [f.n1 for f in fronts]
    g = red.layer_norm_backward(4, 5, [f.dy for f in fronts], [n.h for n in n2], [n.stats for n in n2],
                                [f.params[4] for f in fronts], drop=[f.drops[1] for f in fronts], accumulate=accumulate)
    d = [D.dropout_backward(x.dh + x.dx * 0.5, f.drops[0]) for x, f in zip(g, fronts)]
    g = red.layer_norm_backward(2, 3, d, [n.h for n in n1], [n.stats for n in n1], [f.params[2] for f in fronts],
                                accumulate=accumulate)
    red.embedding_backward(1, [x.dh for x in g], [f.places for f in fronts], accumulate=accumulate)
    red.embedding_backward(0, [x.dh for x in g], [f.tokens for f in fronts], 3.0, accumulate)


def alone(fronts, steps=1):
    out = []
    for f in fronts:
        g = [torch.empty(s, device="cuda") for s in SHAPES]
        f.forward()
        for k in range(steps):
            f.backward(g, accumulate=k > 0)
        out.append(g)
    return out


def mean(rows):
    """Summed in order and divided once, as the reducer does (torch multiplies by
    the reciprocal of a scalar divisor)."""
    s = rows[0].clone()
    for r in rows[1:]:
        s += r
    return s / torch.full_like(s, len(rows))


@pytest.mark.parametrize("views", [False, True])
def test_gradients_through_the_reducer_to_the_step(views):
    R = 3
    fronts, params = replicas(R)
    want = [mean(rows) for rows in zip(*alone(fronts))]
    red = D.Reducer(SHAPES, R, 4 * 2000)
    if views:
        grads = red.bind_bucket_views()
    else:
        grads = [[torch.full(s, 9.0, device="cuda").view(-1) for s in SHAPES] for _ in range(R)]   # flat is fine
        red.bind(grads)
    norm = red.grad_norm()
    opt = red.adamw([[p.clone() for p in params] for _ in range(R)], lr=0.1)
    for it in range(2):
        through_reducer(red, fronts)
        assert [b for b, _ in red.launch_log()] == list(range(red.num_buckets))   # launched before finalize
        red.finalize()
        for v, w in enumerate(want):
            for r in range(R):
                assert torch.equal(grads[r][v].view(SHAPES[v]), w), (it, v, r)
        norm.compute(max_norm=1.0)
        opt.step(clip=norm)
    total = torch.sqrt(sum((w.double() ** 2).sum() for w in want))
    assert abs(float(norm.norm) / float(total) - 1) < 1e-6
    assert opt.steps_done == 2 and not torch.equal(opt.params[0][0], params[0])
    assert torch.equal(opt.params[0][0], opt.params[R - 1][0])


def test_local_steps_through_the_reducer():
    R = 2
    fronts, params = replicas(R, 7)
    want = [mean(rows) for rows in zip(*alone(fronts, 3))]
    red = D.Reducer(SHAPES, R, 1 << 20)
    grads = [[torch.full(s, 9.0, device="cuda") for s in SHAPES] for _ in range(R)]
    red.bind(grads)
    norm = red.grad_norm()
    red.set_sync(False)
    through_reducer(red, fronts)
    through_reducer(red, fronts, accumulate=True)
    with pytest.raises(D.DdpbError) as e:             # local steps that no synchronisation has averaged
        norm.compute()
    assert e.value.code == D.E_STATE
    red.set_sync(True)
    through_reducer(red, fronts, accumulate=True)
    red.finalize()
    for v, w in enumerate(want):
        assert torch.equal(grads[0][v], w) and torch.equal(grads[1][v], w)
    norm.compute()


def test_reducer_refuses_before_it_writes():
    R = 2
    fronts, _ = replicas(R)
    red = D.Reducer(SHAPES, R, 1 << 20)
    toks = [f.tokens for f in fronts]
    d = [f.dy for f in fronts]
    with pytest.raises(D.DdpbError) as e:
        red.embedding_backward(0, d, toks)
    assert e.value.code == D.E_STATE
    grads = [[torch.full(s, 9.0, device="cuda") for s in SHAPES] for _ in range(R)]
    red.bind(grads)
    with pytest.raises(ValueError):
        red.embedding_backward(0, d[:1], toks[:1])    # one replica of two
    with pytest.raises(ValueError):
        red.embedding_backward(2, d, toks)            # no table
    with pytest.raises(D.DdpbError):
        red.embedding_backward(6, d, toks)
    st = [torch.zeros(200, 2, device="cuda")] * R
    with pytest.raises(ValueError):
        red.layer_norm_backward(4, 4, d, d, st)
    with torch.cuda.stream(torch.cuda.Stream()):
        with pytest.raises(ValueError, match="compute stream"):
            red.embedding_backward(0, d, toks)
    with pytest.raises(ValueError):                   # the second replica's: nothing is written for the first
        red.embedding_backward(0, [d[0], d[1][:2]], toks)
    with pytest.raises(ValueError):
        red.layer_norm_backward(4, 5, d, [d[0], d[1][:2]], st)
    assert all((g == 9).all() for row in grads for g in row)
    red.embedding_backward(0, d, toks)
    before = grads[0][0].clone()
    with pytest.raises(D.DdpbError) as e:             # its bucket may be reducing
        red.embedding_backward(0, [2 * x for x in d], toks)
    assert e.value.code == D.E_DOUBLE_READY
    assert torch.equal(grads[0][0], before)
    red.reset()


def test_norm_without_weight_or_bias_through_the_reducer():
    red = D.Reducer([(H,)], 1, 0)
    grads = [[torch.zeros(H, device="cuda")]]
    red.bind(grads)
    h, dy = torch.randn(30, H, device="cuda"), torch.randn(30, H, device="cuda")
    n = D.layer_norm(h)
    red.layer_norm_backward(None, 0, [dy], [h], [n.stats])
    red.finalize()
    assert torch.allclose(grads[0][0], dy.sum(0), atol=1e-4)
    red.layer_norm_backward(None, None, [dy], [h], [n.stats])     # nothing to mark


def test_on_another_stream():
    """Outputs, workspaces and gradients belong to the current stream."""
    tokens, params, dy = inputs(3, n=(40, 64))
    f = Front(tokens, params, dy)
    want = alone([f])[0]
    y = f.forward().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        junk = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):                           # work that the calls have to wait behind
            junk = junk @ junk * 1e-2
        z = f.forward()
        grads = [torch.zeros(sh, device="cuda") for sh in SHAPES]
        f.backward(grads)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(z, y) and all(torch.equal(a, b) for a, b in zip(grads, want))


def test_two_streams_at_once():
    """Two calls at once share no memory: each has a workspace of its own."""
    fronts = [Front(*inputs(20 + i, n=(60, 64))) for i in range(2)]
    want = [alone([f])[0] for f in fronts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in fronts]
    got = [[torch.zeros(sh, device="cuda") for sh in SHAPES] for _ in fronts]
    torch.cuda.synchronize()
    for _ in range(10):
        for f, s, g in zip(fronts, streams, got):
            with torch.cuda.stream(s):
                f.forward()
                f.backward(g)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_captured_and_replayed():
    """A step in a graph: replays follow the inputs and the dropout's counter, the
    same bits as eager calls, with eager calls between the replays."""
    tokens, params, dy = inputs(5)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    f = Front(tokens, params, dy, counter=counter)
    grads = [torch.zeros(s, device="cuda") for s in SHAPES]
    eager = Front(tokens, params, dy, counter=counter)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f.forward()
        f.backward(grads)
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):                                # two graphs, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = f.forward()
            f.backward(grads)
        graphs.append((g, y))
    seen = []
    for k in range(6):
        counter.fill_(10 * k)
        tokens.copy_(torch.randint(-1, VOCAB, tokens.shape, device="cuda"))
        dy.normal_()
        g, y = graphs[k % 2]
        for t in grads:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in grads]
        want = [torch.empty(sh, device="cuda") for sh in SHAPES]
        assert torch.equal(y, eager.forward()), k
        eager.backward(want)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
        seen.append(y.clone())
    assert not any(torch.equal(seen[0], z) for z in seen[1:])


def test_a_sync_captured_behind_them():
    """Backward passes, hooks and the synchronisation in one graph."""
    R = 2
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        fronts, _ = replicas(R, 30)
        red = D.Reducer(SHAPES, R, 4 * 2000)
        grads = [[torch.zeros(sh, device="cuda") for sh in SHAPES] for _ in range(R)]
        red.bind(grads, compute_stream=s)
        through_reducer(red, fronts)
        red.finalize()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        through_reducer(red, fronts)
        red.finalize()
    for k in range(4):
        with torch.cuda.stream(s):
            for f in fronts:
                f.dy.normal_()
            want = [mean(rows) for rows in zip(*alone(fronts))]
            g.replay()
        torch.cuda.synchronize()
        for v, w in enumerate(want):
            assert all(torch.equal(grads[r][v], w) for r in range(R)), (k, v)
    del g
    red.close()


def test_writes_count_for_autograd():
    dw, db, dt = (torch.zeros(s, device="cuda") for s in ((H,), (H,), (VOCAB, H)))
    h = torch.randn(3, H, device="cuda")
    n = D.layer_norm(h)
    v = dw._version, db._version, dt._version
    D.layer_norm_backward(h, h, n.stats, None, dw, db)
    D.embedding_backward(h, torch.arange(3, device="cuda"), dt)
    assert (dw._version, db._version, dt._version) > v and dw._version > v[0] and db._version > v[1]
    assert not n.y.requires_grad


def test_expanded_and_overlapping_inputs():
    row = torch.randn(1, 96, device="cuda")
    x = row.expand(50, 96)
    y = D.layer_norm(x, residual=x).y
    assert torch.equal(y, D.layer_norm((row + row).expand(50, 96).contiguous()).y)
    wide = torch.randn(20, 100, device="cuda")
    sliding = torch.as_strided(wide.view(-1), (50, 40), (7, 1))
    assert torch.equal(D.layer_norm(sliding).y, D.layer_norm(sliding.contiguous()).y)


def test_refusals():
    x, t = torch.randn(4, 8, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    n = D.layer_norm(x)
    bad = [
        lambda: D.layer_norm(x, residual=x[:2]),
        lambda: D.layer_norm(x, residual=x.half()),
        lambda: D.layer_norm(x, weight=x[0, :4]),
        lambda: D.layer_norm(x, weight=x[0], bias=x[0].half()),
        lambda: D.layer_norm(x, weight=x[0].cpu()),
        lambda: D.layer_norm(x.t()),
        lambda: D.layer_norm(x.double()),
        lambda: D.layer_norm(torch.tensor(1.0, device="cuda")),
        lambda: D.layer_norm_backward(x, x[:2], n.stats),
        lambda: D.layer_norm_backward(x, x, n.stats[:2]),
        lambda: D.layer_norm_backward(x, x, n.stats.double()),
        lambda: D.layer_norm_backward(x, x, n.stats, dweight=x[0], dbias=x[1].half()),
        lambda: D.layer_norm_backward(x, x, n.stats, dweight=torch.empty(16, device="cuda")[::2]),
        lambda: D.layer_norm_backward(x, x, n.stats, grad_h=x.bfloat16()),
        lambda: D.dropout(x, D.Drop(0.1, 1), x[0]),
        lambda: D.embedding(t.float(), x), lambda: D.embedding(t.cpu(), x), lambda: D.embedding(t, x[0]),
        lambda: D.embedding(t, x.t()), lambda: D.embedding(t[::2], x), lambda: D.embedding(t, x, residual=x),
        lambda: D.embedding(t, x, dtype=torch.float64),
        lambda: D.embedding_backward(x, t, x.clone()), lambda: D.embedding_backward(x[:3], t, x[:, :4]),
        lambda: D.embedding_backward(x[:3].double(), t, x.clone()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print(i)
    for f in (lambda: D.layer_norm(x, eps=-1.0), lambda: D.embedding(t, x, scale=float("inf")),
              lambda: D.embedding_backward(x[:3], t, x),                       # the gradient of itself
              lambda: D.layer_norm_backward(x, x, n.stats, dweight=x[0])):
        with pytest.raises(D.DdpbError) as e:
            f()
        assert e.value.code == D.E_ARG


@pytest.mark.parametrize("seed", range(12))
def test_random_configurations(seed):
    from layer_util import TYPES, check, make, norm_depth, rows_depth
    g = np.random.default_rng(1000 + seed)
    t = list(TYPES)[seed % 3]
    rows, cols = int(np.exp(g.uniform(0, 7))), int(np.exp(g.uniform(0, 8.5)))
    p, pad = float(g.choice([0.0, 0.1, 0.7])), int(g.choice([0, 1, 6]))
    say(f"random {rows}x{cols} {t} p {p} pad {pad}")
    x, X = make(g, (rows, cols), t, pad)
    r, R = make(g, (rows, cols), t, pad)
    w, W = make(g, (cols,), "f32")
    off = int(g.integers(0, 1 << 62))
    drop, f = D.Drop(p, seed, off), OL.factors((rows, cols), p, seed, off)
    n = D.layer_norm(x, w, None, 1e-3, residual=r, drop=drop)
    z = OL.dropout(X, f, R)
    e = OL.layer_norm_bound(z, OL.dropout_bound(X, f, R), W, None, 1e-3, norm_depth(cols))
    check(n.y, OL.layer_norm(z, W, None, 1e-3)[0], e[0], t, "y")
    m, s = (a.double().cpu().numpy() for a in n.stats[:, :, None].unbind(1))
    H_ = n.h.double().cpu().numpy()
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    out = D.layer_norm_backward(x, n.h, n.stats, w, dw, db, r, drop)
    want = OL.layer_norm_backward(X, H_, m, s, W, R)
    e = OL.layer_norm_backward_bound(X, H_, m, s, W, R, norm_depth(cols), rows_depth(rows))
    for got, a, b, kind in zip((out.dh, dw, db), want, e, (t, "f32", "f32")):
        check(got, a, b, kind, "gradient")
    check(out.dx, OL.dropped(want[0], f), f * e[0] + 2 * OL.U * np.abs(f * want[0]), t, "dx")
