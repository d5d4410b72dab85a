"""Layer norm and the embedding's gradient where a workgroup takes several long rows,
and at the borders between their kernels, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import ddp_bucketed_gradient_amd as D
from gpu_util import require_gpu, say
from oracle import layers as OL
from test_gpu_layers import back_case, grad_case, norm_case, zipf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.synchronize()


# workgroups of the backward pass: at most 256, and 32 to 256 beyond 16384 columns, so that their partial sums stay
# within 64 MiB (40001: 209, 262145: 32); these have more rows than that, and a last turn that not all of them take
@pytest.mark.parametrize("rows, cols", [(300, 4097), (515, 8192), (300, 8195), (600, 16384), (515, 16385), (600, 16391),
                                        (450, 40001), (70, 262145)])
def test_norm_gradient_of_more_long_rows_than_workgroups(rows, cols):
    say(f"norm gradient {rows}x{cols}")
    back_case(rows, rows, cols, "f32", "f32", "f32", False, None, False, 0)
    if cols < 100000:
        back_case(rows + 1, rows, cols, "bf16", "bf16", "bf16", True, 0.1, True, 3)


@pytest.mark.parametrize("t", ["f32", "f16"])
def test_norm_of_more_long_rows_than_workgroups(t):
    """2048 workgroups, a row each at a time: rows do not know of one another."""
    rows, cols = 2048 + 77, 16385
    say(f"norm {rows}x{cols} {t}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(rows, cols, device="cuda", generator=g).to({"f32": torch.float32, "f16": torch.float16}[t])
            for _ in range(2))
    n = D.layer_norm(x, residual=r)
    for a in range(0, rows, 1000):
        b = min(a + 1000, rows)
        part = D.layer_norm(x[a:b], residual=r[a:b])
        assert all(torch.equal(p, q[a:b]) for p, q in zip(part, n))
    norm_case(5, 3, cols, t, "f32", True, 0.1, 0)


@pytest.mark.parametrize("n", [16383, 16384, 16385])
def test_embedding_gradient_at_the_border_of_its_sorts(n):
    g = np.random.default_rng(n)
    for vocab, cols in [(1, 4), (37, 20), (30522, 9)]:
        grad_case(n, zipf(g, n, vocab), vocab, cols, "bf16", "f32", False)
        grad_case(n, g.integers(-1, vocab + 1, n), vocab, cols, "f32", "bf16", True, kind=torch.int32)
    grad_case(n, np.full(n, 30521), 30522, 8, "f32", "f32", True)


# the slices of a row, equal shares of its groups of eight, change where the last would hold one group only: first at
# 4033 groups (32257 columns) and 4097 (32769). A shifted last group is added to with its neighbour, in one wave
@pytest.mark.parametrize("cols", [32249, 32256, 32257, 32263, 32264, 32265, 32769, 32775, 33000])
def test_embedding_gradient_added_to_wide_rows(cols):
    g = np.random.default_rng(cols)
    tokens = np.concatenate([g.integers(-1, 21, 150), np.full(60, 7)])
    for t, gt in (("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")):
        grad_case(cols, tokens, 20, cols, t, gt, True)
    grad_case(cols, tokens, 20, cols, "bf16", "f32", False)


def block_in_64_bits(tokens, table, w1, b1, w2, b2, r, dy, keep):
    """y = drop(norm(r + drop(norm(table[tokens])))) and the gradients of the table, the
    weights and r; the dropouts multiply what they keep by `keep`."""
    leaves = [x.double().cpu().requires_grad_() for x in (table, w1, b1, w2, b2, r)]
    table, w1, b1, w2, b2, r = leaves
    masks = [torch.from_numpy(OL.factors(tuple(dy.shape), 0.1, 11, i)) for i in range(2)]
    m1, m2 = (torch.where(m > 0, k, 0.0) for m, k in zip(masks, keep))

    def norm(z, w, b):
        d = z - z.mean(-1, keepdim=True)
        return d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5) * w + b
    y = norm(r + norm(table[tokens.cpu()], w1, b1) * m1, w2, b2) * m2
    y.backward(dy.double().cpu())
    return [y.detach()] + [x.grad for x in leaves]


def test_a_block_in_bf16_in_the_mean():
    """Against the root of the sum of squares: nine activations and gradients are
    rounded on the way, some of them used twice, each independently and by at most
    2^-8 / sqrt(3) of the value in the mean square; 16 of them, and a factor of two
    for the norms' slopes. The tolerance sees either dropout not scale what it keeps."""
    tol = 2 * 16 ** 0.5 * 2.0 ** -8 / 3 ** 0.5
    g = torch.Generator().manual_seed(3)
    n, vocab, cols = 300, 40, 72
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    tokens = torch.randint(0, vocab, (n,), generator=g).cuda()
    table, w1, b1, w2, b2 = (x.cuda() for x in (rnd(vocab, cols), 1 + 0.3 * rnd(cols), 0.3 * rnd(cols),
                                                1 + 0.3 * rnd(cols), 0.3 * rnd(cols)))
    r, dy = rnd(n, cols).bfloat16().cuda(), rnd(n, cols).bfloat16().cuda()
    drops = [D.Drop(0.1, 11, i) for i in range(2)]
    grads = [torch.full_like(x, float("nan")) for x in (table, w1, b1, w2, b2)]
    n1 = D.layer_norm(D.embedding(tokens, table, dtype=torch.bfloat16), w1, b1)
    n2 = D.layer_norm(n1.y, w2, b2, residual=r, drop=drops[0])
    y = D.dropout(n2.y, drops[1])
    g2 = D.layer_norm_backward(D.dropout_backward(dy, drops[1]), n2.h, n2.stats, w2, grads[3], grads[4], drop=drops[0])
    dz = D.layer_norm_backward(g2.dx, n1.h, n1.stats, w1, grads[1], grads[2]).dh
    D.embedding_backward(dz, tokens, grads[0])
    got = [x.double().cpu() for x in (y, *grads, g2.dh)]

    def off(*keep):
        want = block_in_64_bits(tokens, table, w1, b1, w2, b2, r, dy, keep)
        return max(float((a - b).norm() / b.norm()) for a, b in zip(got, want))
    scale = 65536 / (65536 - OL.limit(0.1))
    assert off(scale, scale) < tol, off(scale, scale)
    for keep in ((1.0, scale), (scale, 1.0)):                       # a mistake in the oracle
        assert off(*keep) > tol, (keep, off(*keep))
