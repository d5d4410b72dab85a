"""The 64-bit oracle of layer norm, dropout and the embedding: published vectors
of the generator, gradients against differences, brute force, and the bounds
against the same formulas in NumPy's float32."""
import numpy as np
import pytest

from oracle import layers as OL

F = np.float32


@pytest.mark.parametrize("counter, key, rounds, want", [
    ([0] * 4, [0] * 2, 10, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, 10, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0], 10,
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]),
    ([0] * 4, [0] * 2, 7, [0x5f6fb709, 0x0d893f64, 0x4f121f81, 0x4f730a48]),
])
def test_generator_gives_its_authors_vectors(counter, key, rounds, want):
    assert OL.philox4x32(counter, key, rounds) == want


def test_random_bits_are_the_words_halves():
    seed, offset = 0x0123456789abcdef, 0xfedcba9876543210
    first, n = (1 << 36) - 5, 21                      # the counter's second word carries
    got = OL.random16(first, n, seed, offset)
    for j in range(n):
        i = first + j
        g = i // 8
        w = OL.philox4x32([g & OL.M32, g >> 32, offset & OL.M32, offset >> 32], [seed & OL.M32, seed >> 32], 7)
        assert got[j] == w[i % 8 // 2] >> 16 * (i % 2) & 0xffff


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9, 1.0, 2.0 ** -16])
def test_share_and_scale(p):
    n = 1 << 18
    f = OL.factors((n,), p, 77, 3)
    kept = (f != 0).sum()
    t = OL.limit(p) / 65536
    assert abs(kept - (1 - t) * n) <= 5 * np.sqrt(n * t * (1 - t)) + 1e-9
    assert p == 1.0 or np.allclose(f[f != 0], 1 / (1 - t), rtol=1e-15)
    x = np.full(n, np.inf)
    y = OL.dropout(x, f)
    assert np.isposinf(y[f != 0]).all() and (y[f == 0] == 0).all()


def _norm_of(x, w, b, eps, r, f):
    return OL.layer_norm(OL.dropout(x, f, r), w, b, eps)[0]


@pytest.mark.parametrize("rows, cols", [(3, 5), (2, 1), (4, 16)])
def test_norm_gradients_against_differences(rows, cols):
    g = np.random.default_rng(rows * 100 + cols)
    x, r, c, more = (g.normal(size=(rows, cols)) for _ in range(4))
    w, b, eps = g.normal(size=cols), g.normal(size=cols), 1e-3
    f = OL.factors((rows, cols), 0.25, 5, 6)
    h = OL.dropout(x, f, r)
    _, mean, rstd = OL.layer_norm(h, w, b, eps)
    dh, dw, db = OL.layer_norm_backward(c, h, mean, rstd, w, more)
    loss = lambda x, r, w, b: (_norm_of(x, w, b, eps, r, f) * c).sum() + (OL.dropout(x, f, r) * more).sum()  # noqa: E731
    for name, at, grad in (("x", 0, OL.dropped(dh, f)), ("r", 1, dh), ("w", 2, dw), ("b", 3, db)):
        args = [x, r, w, b]
        for i in np.ndindex(grad.shape):
            e = np.zeros_like(args[at])
            e[i] = 1e-6
            up, down = list(args), list(args)
            up[at], down[at] = args[at] + e, args[at] - e
            want = (loss(*up) - loss(*down)) / 2e-6
            # of the difference: 2^-53 * |loss| / 1e-6 from rounding, the third derivative times 1e-12
            assert abs(grad[i] - want) < 2e-6 * (1 + abs(want)), (name, i)


def test_embedding_gradient_against_differences():
    g = np.random.default_rng(0)
    table, c = g.normal(size=(6, 3)), g.normal(size=(9, 3))
    tokens = [1, 4, 1, -1, 6, 0, 1, 5, 4]
    d = OL.embedding_backward(c, tokens, 6, 0.5)
    for i in np.ndindex(table.shape):
        e = np.zeros_like(table)
        e[i] = 1.0                                    # linear: any step will do
        assert abs((OL.embedding(tokens, e, 0.5) * c).sum() - d[i]) < 1e-14
    assert (d[2] == 0).all() and (d[3] == 0).all()
    assert (OL.embedding(tokens, table)[[3, 4]] == 0).all()


@pytest.mark.parametrize("seed", range(6))
def test_bounds_hold_for_float32(seed):
    """NumPy's float32 sums pairwise in blocks of 128 elements (8 of them side by
    side): at most 16 + 3 + log2(cols / 128) additions deep."""
    g = np.random.default_rng(seed)
    rows, cols = 7, int(g.integers(1, 3000))
    depth = 20 + 8
    x = (g.normal(size=(rows, cols)) * 10.0 ** g.integers(-3, 4) + g.normal() * 10).astype(F)
    r = g.normal(size=(rows, cols)).astype(F)
    w, b, eps = g.normal(size=cols).astype(F), g.normal(size=cols).astype(F), 1e-5
    f = OL.factors((rows, cols), 0.1, seed, 1)
    z = np.where(f == 0, F(0), x * F(65536 / (65536 - OL.limit(0.1)))) + r
    mean = z.mean(1, keepdims=True, dtype=F)
    d = z - mean
    rstd = F(1) / np.sqrt((d * d).mean(1, keepdims=True, dtype=F) + F(eps))
    y = d * rstd * w + b
    X, R, W, B = (a.astype(np.float64) for a in (x, r, w, b))
    Z = OL.dropout(X, f, R)
    Y, M, S = OL.layer_norm(Z, W, B, eps)
    e_y, e_m, e_s = OL.layer_norm_bound(Z, OL.dropout_bound(X, f, R), W, B, eps, depth)
    e_y = e_y + OL.U * np.abs(W * (Z - M) * S)        # the product is rounded before the sum here
    for got, want, bound in ((y, Y, e_y), (mean, M, e_m), (rstd, S, e_s)):
        assert (np.abs(got - want) <= 1.01 * bound).all()
    dy = g.normal(size=(rows, cols)).astype(F)
    n = (z - mean) * rstd
    k = dy * w
    dh = rstd * (k - k.mean(1, keepdims=True, dtype=F) - n * (k * n).mean(1, keepdims=True, dtype=F))
    want = OL.layer_norm_backward(dy.astype(float), z.astype(float), mean.astype(float), rstd.astype(float), W)
    bound = OL.layer_norm_backward_bound(dy.astype(float), z.astype(float), mean.astype(float), rstd.astype(float), W,
                                         None, depth, rows)
    for got, a, e in zip((dh, (dy * n).sum(0, dtype=F), dy.sum(0, dtype=F)), want, bound):
        assert (np.abs(got - a) <= 1.01 * e + 1e-30).all()


def test_planted_mistakes_are_outside_of_the_bounds():
    g = np.random.default_rng(9)
    z, w, dy = g.normal(size=(4, 64)), g.normal(size=64), g.normal(size=(4, 64))
    y, mean, rstd = OL.layer_norm(z, w)
    e = OL.layer_norm_bound(z, 0 * z, w, None, 1e-5, 32)
    wrong = OL.layer_norm(z, w, None, 1e-5 * 1.01 + z.var(1).mean() / 64)[0]       # cols - 1 in place of cols
    assert (np.abs(wrong - y) > e[0] + OL.rounding(y, "f32")).mean() > 0.9
    dh, dw, db = OL.layer_norm_backward(dy, z, mean, rstd, w)
    e = OL.layer_norm_backward_bound(dy, z, mean, rstd, w, None, 32, 32)
    no_mean = rstd * (dy * w - ((z - mean) * rstd) * (dy * w * (z - mean) * rstd).mean(1, keepdims=True))
    assert (np.abs(no_mean - dh) > e[0]).mean() > 0.9
