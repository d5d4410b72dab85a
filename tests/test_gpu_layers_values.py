"""Layer norm's gradients where values are far out: rows that are nearly constant at
a large mean, as masks and saturated channels leave them."""
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


@pytest.mark.parametrize("cols", [1, 2, 3, 7, 8, 9, 20, 64, 100, 127, 256, 300, 520, 1000, 1100, 2049, 3000, 4100, 8200,
                                  16390])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_mean_times_rstd_beyond_fp32(cols, t):
    """(0 - mean) rstd overflows, which no column that exists computes."""
    rows = 5
    say(f"large mean {rows}x{cols} {t}")
    g = np.random.default_rng(cols)
    mean, rstd = 2.0 ** 110, 2.0 ** 20
    h = torch.full((rows, cols), mean, dtype=TYPES[t], device="cuda")
    H = np.full((rows, cols), mean)
    dy, DY = make(g, (rows, cols), t)
    w, W = make(g, (cols,), "f32")
    stats = torch.tensor([[mean, rstd]] * rows, device="cuda")
    m, s = np.full((rows, 1), mean), np.full((rows, 1), rstd)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    out = D.layer_norm_backward(dy, h, stats, w, dw, db)
    want = OL.layer_norm_backward(DY, H, m, s, W)
    bound = OL.layer_norm_backward_bound(DY, H, m, s, W, None, norm_depth(cols), rows_depth(rows))
    for got, a, b, kind in zip((out.dh, dw, db), want, bound, (t, "f32", "f32")):
        check(got, a, b, kind, "gradient")


@pytest.mark.parametrize("cols", [1, 4, 8, 64, 256])
def test_constant_rows_at_a_large_mean_both_ways(cols):
    # 2^k values of 2^115: their sum is at most 2^123 (256 of 2^120 would be 2^128, beyond fp32) and, like the mean,
    # exact; rstd = 10^4.5 > 2^14, so mean * rstd is beyond 2^128
    x = torch.full((3, cols), 2.0 ** 115, device="cuda")
    n = D.layer_norm(x, eps=1e-9)
    assert (n.y == 0).all() and (n.stats[:, 0] == 2.0 ** 115).all()
    dy = torch.arange(cols, device="cuda").float().expand(3, cols)
    dh = D.layer_norm_backward(dy, x, n.stats).dh
    want = (dy - dy.mean(1, keepdim=True)) * n.stats[:, 1:]
    assert torch.allclose(dh, want, rtol=1e-6, atol=0)
