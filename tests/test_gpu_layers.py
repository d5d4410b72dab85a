"""Layer norm, dropout and the embedding against the 64-bit oracle, element by
element, within bounds derived from the number of fp32 roundings."""
import numpy as np
import pytest
import torch

import ddp_bucketed_gradient_amd as D
from gpu_util import require_gpu, say
from layer_util import TYPES, check, make, norm_depth, rows_depth
from oracle import layers as OL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.synchronize()


def norm_case(seed, rows, cols, t, w, residual, p, pad, eps=1e-5, shift=0.5, scale=1.0):
    g = np.random.default_rng(seed)
    x, X = make(g, (rows, cols), t, pad, scale, shift)
    r, R = make(g, (rows, cols), t, pad) if residual else (None, None)
    wt, W = make(g, (cols,), w) if w else (None, None)
    b, B = make(g, (cols,), w) if w else (None, None)
    drop = D.Drop(p, seed + 1, 7) if p is not None else None
    f = OL.factors((rows, cols), p or 0.0, seed + 1, 7)
    n = D.layer_norm(x, wt, b, eps, residual=r, drop=drop)
    z = OL.dropout(X, f, R)
    z_err = OL.dropout_bound(X, f, R) if residual or OL.limit(p or 0) else 0 * z
    e_y, e_m, e_s = OL.layer_norm_bound(z, z_err, W, B, eps, norm_depth(cols))
    y, m, s = OL.layer_norm(z, W, B, eps)
    check(n.stats[..., 0], m[:, 0], e_m[:, 0], "f32", "mean")
    check(n.stats[..., 1], s[:, 0], e_s[:, 0], "f32", "rstd")
    check(n.y, y, e_y, t, "y")
    if residual or OL.limit(p or 0):
        check(n.h, z, z_err, t, "h")
    else:
        assert n.h is x


COLS = [1, 2, 7, 8, 9, 16, 64, 127, 128, 129, 511, 512, 513, 768, 771, 1024, 1025, 2047, 2048, 2056, 4096, 4097, 8192,
        8195, 16384, 16391, 40001]


@pytest.mark.parametrize("i, cols", list(enumerate(COLS)))
def test_norm_every_shape(i, cols):
    rows = [1, 3, 17, 70, 5][i % 5] if cols < 2000 else 3
    t = ["f32", "bf16", "f16"][i % 3]
    say(f"norm {rows}x{cols} {t}")
    norm_case(i, rows, cols, t, ["f32", t][i // 3 % 2], False, None, 0)
    norm_case(i + 100, rows, cols, t, t, True, 0.1, [0, 3, 8][i // 2 % 3])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("w, residual, p", [(None, False, None), ("f32", True, None), ("bf16", False, 0.5),
                                            ("f16", True, 0.0), ("f32", True, 1.0), (None, True, 0.9)])
def test_norm_every_input(t, w, residual, p):
    for rows, cols, pad in [(9, 96, 0), (5000, 40, 1), (31, 777, 5), (6, 1031, 0)]:
        say(f"norm {rows}x{cols} {t} weights {w} residual {residual} p {p}")
        norm_case(3, rows, cols, t, w, residual, p, pad)


def test_norm_large_mean_and_constant_rows():
    norm_case(1, 4, 1000, "f32", "f32", False, None, 0, shift=1000.0, scale=0.1)
    norm_case(2, 4, 1000, "f32", "f32", False, None, 0, shift=0.0, scale=1e-12)
    x = torch.full((3, 50), 2.5, device="cuda")
    n = D.layer_norm(x, eps=1e-5)
    assert (n.y == 0).all() and (n.stats[:, 0] == 2.5).all()
    n = D.layer_norm(x, eps=0.0)                      # 0 / 0, as the formula says
    assert n.y.isnan().all() and n.stats[:, 1].isinf().all()


def test_norm_rows_that_are_not_finite_stay_alone():
    x = torch.randn(6, 300, device="cuda")
    want = D.layer_norm(x).y.clone()
    x[1, 5], x[4, 299] = float("inf"), float("nan")
    got = D.layer_norm(x).y
    assert torch.equal(got[[0, 2, 3, 5]], want[[0, 2, 3, 5]]) and got[[1, 4]].isnan().all()


def back_case(seed, rows, cols, t, w, gt, more, p, add, pad):
    g = np.random.default_rng(seed)
    h, H = make(g, (rows, cols), t, pad, shift=0.3)
    dy, DY = make(g, (rows, cols), t, pad and pad + 1)
    gh, GH = make(g, (rows, cols), t) if more else (None, None)
    wt, W = make(g, (cols,), w) if w else (None, None)
    dw, DW = make(g, (cols,), gt)
    db, DB = make(g, (cols,), gt)
    _, m, s = OL.layer_norm(H)
    stats = torch.from_numpy(np.concatenate([m, s], 1)).float().cuda()
    m, s = (x.cpu().numpy() for x in stats.double()[:, :, None].unbind(1))
    drop = D.Drop(p, seed, 1 << 40) if p is not None else None
    out = D.layer_norm_backward(dy, h, stats, wt, dw, db, gh, drop, add)
    dh, dW, dB = OL.layer_norm_backward(DY, H, m, s, W, GH)
    e_h, e_w, e_b = OL.layer_norm_backward_bound(DY, H, m, s, W, GH, norm_depth(cols), rows_depth(rows))
    check(out.dh, dh, e_h, t, "dh")
    f = OL.factors((rows, cols), p or 0.0, seed, 1 << 40)
    if OL.limit(p or 0):
        check(out.dx, OL.dropped(dh, f), f * e_h + 2 * OL.U * np.abs(f * dh), t, "dx")
    else:
        assert out.dx is out.dh
    # adding to the old value rounds once more
    check(dw, dW + DW * add, e_w + add * OL.U * np.abs(dW + DW), gt, "dweight")
    check(db, dB + DB * add, e_b + add * OL.U * np.abs(dB + DB), gt, "dbias")


@pytest.mark.parametrize("i, cols", list(enumerate(COLS)))
def test_norm_gradient_every_shape(i, cols):
    rows = [1, 3, 17, 70, 4200][i % 5] if cols < 600 else [1, 5, 1300][i % 3] if cols < 2000 else 3
    t = ["bf16", "f32", "f16"][i % 3]
    say(f"norm gradient {rows}x{cols} {t}")
    back_case(i, rows, cols, t, "f32", "f32", False, None, False, 0)
    back_case(i + 50, rows, cols, t, t, ["f32", t][i % 2], True, 0.25, True, [0, 3, 8][i // 2 % 3])


@pytest.mark.parametrize("rows", [513, 2048, 4097, 9000])
def test_norm_gradient_many_rows(rows):
    back_case(rows, rows, 65, "f32", "f32", "f32", False, None, False, 0)
    back_case(rows, rows, 530, "bf16", "bf16", "bf16", True, 0.1, True, 1)
    back_case(rows, rows, 2050, "f16", None, "f32", False, None, False, 0)


@pytest.mark.parametrize("rows, cols", [(128, 100), (129, 100), (4, 128), (32, 1000), (33, 1000), (4, 2001), (5, 2001),
                                        (4, 8003), (1, 16384), (5, 16384)])
def test_norm_gradient_by_one_workgroup_and_by_more(rows, cols):
    back_case(rows, rows, cols, "f32", "f32", "f32", False, None, False, 0)
    back_case(rows, rows, cols, "bf16", "f32", "bf16", True, 0.1, True, 3)


@pytest.mark.parametrize("rows, cols", [(40, 100), (400, 100), (3, 5000)])
def test_norm_gradient_parts_that_are_not_wanted(rows, cols):
    g = np.random.default_rng(0)
    h, _ = make(g, (rows, cols), "f32")
    dy, _ = make(g, (rows, cols), "f32")
    n = D.layer_norm(h)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    full = D.layer_norm_backward(dy, h, n.stats, None, dw, db)
    for a, b in ((torch.empty_like(dw), None), (None, torch.empty_like(db)), (None, None)):
        out = D.layer_norm_backward(dy, h, n.stats, None, a, b)
        assert torch.equal(out.dh, full.dh)
        assert (a is None or torch.equal(a, dw)) and (b is None or torch.equal(b, db))


def test_no_rows():
    w = torch.ones(7, device="cuda")
    n = D.layer_norm(torch.empty(0, 7, device="cuda"), w, w)
    assert n.y.shape == (0, 7) and n.stats.shape == (0, 2)
    dw, db = torch.full((7,), 3.0, device="cuda"), torch.full((7,), 4.0, device="cuda")
    D.layer_norm_backward(n.y, n.h, n.stats, w, dw, db, accumulate=True)
    assert (dw == 3).all() and (db == 4).all()
    D.layer_norm_backward(n.y, n.h, n.stats, w, dw, db)
    assert (dw == 0).all() and (db == 0).all()
    for shape in ((0, 5), (5, 0), (0,)):
        assert D.dropout(torch.empty(shape, device="cuda"), D.Drop(0.1, 1)).shape == shape
    with pytest.raises(D.DdpbError):
        D.layer_norm(torch.empty(3, 0, device="cuda"))


# ---- dropout --------------------------------------------------------------------

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shape, pad", [((1,), 0), ((7,), 0), ((8,), 0), ((1, 9), 0), ((20, 10), 0), ((3, 5, 17), 0),
                                        ((4100, 33), 0), ((37, 8), 8), ((300, 7), 1), ((2049, 153), 3), ((2, 70001), 5),
                                        ((3, 4, 64), 2)])
def test_dropout(t, shape, pad):
    g = np.random.default_rng(len(shape) * 100 + shape[-1])
    for p, residual, seed, offset in [(0.1, False, 1, 0), (0.5, True, -3, 1 << 63), (0.0, True, 1, 1), (1.0, True, 2, 2)]:
        say(f"dropout {shape} +{pad} {t} p {p}")
        x, X = make(g, shape, t, pad if len(shape) < 3 or pad == 0 else 0)
        r, R = make(g, shape, t, pad + 2 if pad and len(shape) < 3 else 0) if residual else (None, None)
        f = OL.factors(shape, p, seed, offset)
        y = D.dropout(x, D.Drop(p, seed, offset), r)
        check(y, OL.dropout(X, f, R), OL.dropout_bound(X, f, R), t, "y")
        if not residual:
            assert torch.equal(D.dropout_backward(x, D.Drop(p, seed, offset)), y)


def test_dropout_hides_what_it_drops():
    x = torch.full((64, 100), float("nan"), device="cuda")
    r = torch.ones_like(x)
    f = torch.from_numpy(OL.factors((64, 100), 0.3, 9, 4)).cuda()
    y = D.dropout(x, D.Drop(0.3, 9, 4), r)
    assert torch.equal(y.isnan(), f != 0) and (y[f == 0] == 1).all()
    assert (D.dropout(x, D.Drop(1.0, 9, 4)) == 0).all()


@pytest.mark.parametrize("rows, cols, pad", [(1, 1000, 0), (37, 19, 0), (37, 19, 4), (300, 7, 1), (50, 771, 2), (9, 64, 8), (2049, 13, 3)])
def test_dropout_in_place(rows, cols, pad):
    """Through the C call, which allows y to be x or the residual."""
    lib = D.lib()
    stream = torch.cuda.current_stream().cuda_stream
    for t in TYPES:
        g = np.random.default_rng(cols)
        x, _ = make(g, (rows, cols), t)
        other, _ = make(g, (rows, cols), t, pad)
        drop = D.Drop(0.4, 6, 7)
        want = D.dropout(x, drop, other)
        y = x.clone()
        lib.dropout(rows, cols, {"f32": D.F32, "bf16": D.BF16, "f16": D.F16}[t], y.data_ptr(), cols, other.data_ptr(),
                    other.stride(0), drop._c, y.data_ptr(), stream)
        assert torch.equal(y, want)
        y = x.clone()                                  # onto the residual
        want = D.dropout(other, drop, x)
        lib.dropout(rows, cols, {"f32": D.F32, "bf16": D.BF16, "f16": D.F16}[t], other.data_ptr(), other.stride(0),
                    y.data_ptr(), cols, drop._c, y.data_ptr(), stream)
        assert torch.equal(y, want)


def test_dropout_counter_is_added_to_the_offset():
    x = torch.randn(1000, device="cuda")
    c = torch.tensor([5], device="cuda")
    assert torch.equal(D.dropout(x, D.Drop(0.5, 3, 10, c)), D.dropout(x, D.Drop(0.5, 3, 15)))
    c.fill_(-11)                                      # the sum wraps
    assert torch.equal(D.dropout(x, D.Drop(0.5, 3, 10, c)), D.dropout(x, D.Drop(0.5, 3, -1)))


def test_norms_dropout_is_dropouts():
    """The fused h is dropout's output bit for bit, and its gradient dropout's."""
    for cols in (64, 100, 771, 1024, 5000):
        x, r, dy = (torch.randn(50, cols, device="cuda", dtype=torch.bfloat16) for _ in range(3))
        d = D.Drop(0.2, 8, 123)
        n = D.layer_norm(x, residual=r, drop=d)
        assert torch.equal(n.h, D.dropout(x, d, r))
        x32, r32 = x.float(), r.float()
        n = D.layer_norm(x32, residual=r32, drop=d)
        assert torch.equal(n.y, D.layer_norm(D.dropout(x32, d, r32)).y)
        out = D.layer_norm_backward(dy.float(), n.h, n.stats, drop=d)
        assert torch.equal(out.dx, D.dropout_backward(out.dh, d))


# ---- embedding ------------------------------------------------------------------

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("w", TYPES)
def test_lookup(t, w):
    g = np.random.default_rng(5)
    for n, vocab, cols in [(1, 1, 1), (3, 10, 7), (1000, 50, 8), (17, 512, 100), (260, 1000, 771), (5, 3, 4099)]:
        table, T = make(g, (vocab, cols), w)
        tokens = g.integers(-2, vocab + 2, n)
        tokens[0] = vocab - 1
        for kind in (torch.int64, torch.int32):
            r, R = make(g, (n, cols), t, 3) if kind is torch.int32 else (None, None)
            y = D.embedding(torch.from_numpy(tokens).to(kind).cuda(), table, 0.7, r, TYPES[t])
            check(y, OL.embedding(tokens, T, 0.7, R), OL.embedding_bound(tokens, T, 0.7, R), t, f"{n} {vocab} {cols}")


def test_lookup_far_tokens_and_shapes():
    table = torch.randn(4, 3, device="cuda")
    tokens = torch.tensor([[0, 1 << 32, -1], [(1 << 63) - 1, -(1 << 63), 3]], device="cuda")
    y = D.embedding(tokens, table)
    assert y.shape == (2, 3, 3) and torch.equal(y[0, 0], table[0]) and torch.equal(y[1, 2], table[3])
    assert (y[0, 1:] == 0).all() and (y[1, :2] == 0).all()
    assert D.embedding(tokens[:, :0].contiguous(), table).shape == (2, 0, 3)
    assert (D.embedding(tokens, table[:0]) == 0).all()


def grad_case(seed, tokens, vocab, cols, t, gt, add, pad=0, scale=0.5, kind=torch.int64):
    g = np.random.default_rng(seed)
    tokens = np.asarray(tokens, dtype=np.int64)
    n = len(tokens)
    say(f"embedding gradient n {n} vocab {vocab} cols {cols} {t} {gt} add {add}")
    dy, DY = make(g, (n, cols), t, pad)
    d, OLD = make(g, (vocab, cols), gt)
    out = D.embedding_backward(dy, torch.from_numpy(tokens).to(kind).cuda(), d, scale, add)
    assert out is d
    want, bound = OL.embedding_backward(DY, tokens, vocab, scale), OL.embedding_backward_bound(DY, tokens, vocab, scale)
    check(d, want + OLD * add, bound + add * OL.U * np.abs(want + OLD), gt, "dtable")
    if add:                                           # rows of no token: the same bits
        rest = np.setdiff1d(np.arange(vocab), tokens)
        assert np.array_equal(d.double().cpu().numpy()[rest], OLD[rest])


def zipf(g, n, vocab):
    return np.minimum(np.exp(g.random(n) * np.log(vocab + 1)).astype(np.int64), vocab) - 1


@pytest.mark.parametrize("i, n", list(enumerate([0, 1, 2, 7, 8, 9, 63, 64, 65, 1000, 4095, 4096, 4097, 8192, 12289])))
def test_gradient_lengths(i, n):
    g = np.random.default_rng(n)
    t, gt = ["f32", "bf16", "f16"][i % 3], ["f32", "f32", "f16", "bf16"][i % 4]
    for vocab, cols in [(1, 3), (37, 20), (1023, 8), (1024, 65), (5000, 5)]:
        grad_case(i, g.integers(-1, vocab + 1, n), vocab, cols, t, gt, i % 2 == 1, pad=i % 3)
        grad_case(i, zipf(g, n, vocab), vocab, cols, t, "f32", i % 2 == 0, kind=torch.int32)


@pytest.mark.parametrize("cols", [1, 8, 60, 64, 65, 512, 513, 768, 1024, 2049, 4100])
def test_gradient_widths(cols):
    g = np.random.default_rng(cols)
    tokens = zipf(g, 600, 300)
    tokens[100:180] = 4
    grad_case(1, tokens, 300, cols, "bf16", "f32", False)
    grad_case(2, tokens, 300, cols, "f32", "bf16", True, pad=3)


@pytest.mark.parametrize("name, tokens", [
    ("one token", np.full(3000, 3)),
    ("one token, many tiles", np.full(20000, 3)),
    ("all outside", np.full(5000, -1)),
    ("last token and outside", np.repeat([40, 39, 41], 2000)),
    ("each once", np.arange(41)),
    ("runs of a unit", np.repeat(np.arange(41), 8)),
    ("runs of a unit, one off", np.concatenate([[0], np.repeat(np.arange(41), 8)])),
    ("runs of nearly two units", np.repeat(np.arange(41), 14)),
    ("runs of two units", np.repeat(np.arange(41), 16)),
    ("one long run among short ones", np.concatenate([np.arange(13), np.full(500, 20), np.arange(14, 41)])),
    ("a run to the end", np.concatenate([np.arange(5), np.full(100, 30)])),
    ("two long runs meet", np.concatenate([np.full(1003, 7), np.full(1005, 8)])),
    ("shuffled", np.random.default_rng(0).permutation(np.repeat(np.arange(41), 300))),
])
@pytest.mark.parametrize("add", [False, True])
def test_gradient_runs(name, tokens, add):
    grad_case(1, tokens, 41, 24, "f32", "f32", add)
    grad_case(2, np.random.default_rng(1).permutation(tokens), 41, 600, "bf16", "bf16", add)


@pytest.mark.parametrize("n, vocab", [(262144, 300), (262145, 30522), (300001, (1 << 20) + 7), (5000, (1 << 20) + 7),
                                      (70000, 2000), (3000, (1 << 21) - 1)])
def test_gradient_many_tiles_and_passes(n, vocab):
    g = np.random.default_rng(n)
    tokens = zipf(g, n, vocab)
    tokens[g.random(n) < 0.3] = vocab - 1
    grad_case(3, tokens, vocab, 3, "f32", "f32", False)
    grad_case(4, g.integers(0, vocab, n), vocab, 2, "f16", "f16", True)


def test_gradient_millions_of_places():
    """Units longer than 128 places, thousands of tiles, a run of half of the places."""
    g = np.random.default_rng(3)
    n, vocab = 9_000_001, 1000
    tokens = g.integers(-1, vocab + 1, n)
    tokens[g.random(n) < 0.5] = 77
    dy, DY = make(g, (n, 1), "f32")
    d, OLD = make(g, (vocab, 1), "f32")
    D.embedding_backward(dy, torch.from_numpy(tokens).cuda(), d, 0.25, True)
    inside = (tokens >= 0) & (tokens < vocab)
    sums = lambda x: np.bincount(tokens[inside], x[inside, 0], vocab)[:, None]  # noqa: E731
    want = 0.25 * sums(DY)
    # deep: a unit's places one after the other (256), then the parts of the longest run, 4.5 M / 256 over 16 lanes
    bound = (256 + 3 + 4_600_000 // 256 // 16 + 16) * OL.U * 0.25 * sums(np.abs(DY)) + OL.U * np.abs(want + OLD)
    check(d, want + OLD, bound, "f32", "dtable")


@pytest.mark.parametrize("offset", [0, 1, 3, 7])
@pytest.mark.parametrize("gt", ["f32", "bf16"])
def test_gradient_at_odd_addresses(offset, gt):
    """A table inside a larger storage: nothing around it is written."""
    for vocab, cols in [(1, 1), (3, 1), (2, 7), (50, 33), (4000, 17)]:
        flat = torch.full((offset + vocab * cols + 9,), 5.0, dtype=TYPES[gt], device="cuda")
        d = flat[offset:offset + vocab * cols].view(vocab, cols)
        tokens = torch.arange(0, vocab, 2, device="cuda")
        dy = torch.ones(len(tokens), cols, dtype=TYPES[gt], device="cuda")
        D.embedding_backward(dy, tokens, d)
        want = (torch.arange(vocab, device="cuda") % 2 == 0).to(TYPES[gt])[:, None].expand(vocab, cols)
        assert torch.equal(d, want)
        assert (flat[:offset] == 5).all() and (flat[offset + vocab * cols:] == 5).all()


def test_same_bits_on_every_run():
    g = np.random.default_rng(0)
    tokens = torch.from_numpy(zipf(g, 30000, 3000)).cuda()
    dy = torch.randn(30000, 256, device="cuda", dtype=torch.bfloat16)
    h, d2 = torch.randn(9000, 640, device="cuda"), torch.randn(9000, 640, device="cuda")
    n = D.layer_norm(h)
    first = None
    for _ in range(4):
        d = D.embedding_backward(dy, tokens, torch.empty(3000, 256, device="cuda"))
        dw, db = torch.empty(640, device="cuda"), torch.empty(640, device="cuda")
        D.layer_norm_backward(d2, h, n.stats, None, dw, db)
        now = [x.clone() for x in (d, dw, db)]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(now, first))


# ---- beyond 32 bits -------------------------------------------------------------

def test_more_than_2_to_the_31_elements():
    cols, rows = 4096, (1 << 19) + 37                 # 2^31 elements and some
    say("more than 2^31 elements: dropout")
    x = torch.ones(rows, cols, dtype=torch.float16, device="cuda")
    x[-1] = torch.arange(cols, device="cuda") * 0.01
    d = D.Drop(0.5, 4, 2)
    y = D.dropout(x, d)
    keep = OL.random16((rows - 2) * cols, 2 * cols, 4, 2) >= 32768
    want = x[-2:].double().cpu().numpy() * 2 * keep.reshape(2, cols)
    check(y[-2:], want, 0 * want, "f16", "dropout")
    del y
    say("more than 2^31 elements: norm")
    n = D.layer_norm(x)
    z = x[-1:].double().cpu().numpy()
    want = OL.layer_norm(z)
    bound = OL.layer_norm_bound(z, 0 * z, None, None, 1e-5, norm_depth(cols))
    check(n.y[-1:], want[0], bound[0], "f16", "norm")
    out = D.layer_norm_backward(n.y, x, n.stats)
    assert out.dh.shape == x.shape and (out.dh[:-1] == 0).all()
    del out, n, x
    say("more than 2^31 elements: embedding")
    vocab = (1 << 30) + 11
    d = torch.full((vocab, 2), 7.0, dtype=torch.bfloat16, device="cuda")
    tokens = torch.tensor([vocab - 1, 5, vocab - 1, 1 << 30], device="cuda")
    dy = torch.tensor([[1.0, 2], [3, 4], [5, 6], [7, 8]], device="cuda")
    D.embedding_backward(dy, tokens, d, accumulate=True)
    assert d[[vocab - 1, 1 << 30, 5, vocab - 2]].tolist() == [[13, 15], [14, 15], [10, 11], [7, 7]]
    assert D.embedding(tokens, d).tolist() == [[13, 15], [10, 11], [13, 15], [14, 15]]
    D.embedding_backward(dy, tokens, d)
    assert d[[vocab - 1, 1 << 30, 5]].tolist() == [[6, 8], [7, 8], [3, 4]]
    assert int((d != 0).any(1).sum()) == 3
