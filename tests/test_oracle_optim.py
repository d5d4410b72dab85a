"""The 64-bit oracle of the optimizer step, pinned by closed forms, by torch's
float8 types and by statistics of its rounding."""
import math

import numpy as np
import pytest
import torch

from oracle import optim as OO


def test_norm_of_known_triangles():
    assert OO.norm([np.array([3.0]), np.array([4.0])]) == 5.0
    assert OO.norm([np.array([3.0]), np.array([4.0])], grad_scale=-0.5) == 2.5
    assert OO.norm([]) == 0.0
    assert OO.norm([np.array([3e30]), np.array([4e30])]) == pytest.approx(5e30, rel=1e-15)
    assert math.isinf(OO.norm([np.array([1.0, -np.inf])])) and math.isnan(OO.norm([np.array([np.inf, np.nan])]))
    assert OO.clip_coef(5.0, 1.0) == 0.2 and OO.clip_coef(0.5, 1.0) == 1.0 and OO.clip_coef(1.0, 1.0) == 1.0


def test_adamw_against_torch_in_fp64():
    rng = np.random.default_rng(1)
    w0, gs = rng.normal(size=50), rng.normal(size=(5, 50))
    p = torch.nn.Parameter(torch.from_numpy(w0.copy()))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    w, m, v = w0, np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        p.grad = torch.from_numpy(gs[t - 1])
        opt.step()
        (w, m, v, _), _ = OO.adamw(w, gs[t - 1], m, v, t=t, lr=3e-3, beta1=0.8, beta2=0.95, eps=1e-6,
                                   weight_decay=0.1, gscale=1.0)
        # Both round each of at most 16 operations of a step to 2^-53 of terms
        # no larger than |w| along the way (|w0| plus at most 5 updates of lr |m| /
        # (1 - 0.8^t) / (sqrt(v) / sqrt(1 - 0.95^t)) < 1.5 lr here): 5 steps, two
        # sides. Relative to w alone nothing holds, as w may pass through 0.
        atol = 2 * 5 * 16 * 2.0 ** -53 * (np.abs(w0) + 5 * 1.5 * 3e-3)
        assert (np.abs(w - p.detach().numpy()) <= atol).all()


def test_the_first_step_is_the_sign_of_the_gradient():
    """t = 1 from a zero state: m / (1 - beta1) = g and v / (1 - beta2) = g^2."""
    g = np.array([2.0, -0.5, 1e-3])
    (w, _, _, _), _ = OO.adamw(np.zeros(3), g, np.zeros(3), np.zeros(3), t=1, lr=0.1, beta1=0.9, beta2=0.999, eps=0.0,
                               weight_decay=0.0, gscale=1.0)
    np.testing.assert_allclose(w, -0.1 * np.sign(g), rtol=1e-12)


def test_code_values_are_torchs_e4m3():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(OO.CODES, want)


@pytest.mark.parametrize("top,s", [(448.0, 127), (448.0000001, 128), (1.75, 119), (1.75001, 120), (1.0, 119),
                                   (0.875, 118), (2.0 ** -120, 1), (1e-300, 1), (0.0, 1), (3e38, 247)])
def test_scales(top, s):
    x = np.zeros(65)
    x[3] = -top
    assert OO.scales_of(x).tolist() == [s, 1]


def test_scales_leave_out_what_is_not_finite():
    x = np.array([1.0, np.inf, np.nan, -np.inf])
    assert OO.scales_of(x).tolist() == [119]


def test_rounding_is_unbiased_and_uses_neighbouring_codes():
    """A value a quarter of a step above a code rounds up in a quarter of all
    cases: over n independent draws within 5 standard deviations."""
    n = 1 << 16
    um, ur = OO.random16(12345, 7, np.arange(n, dtype=np.uint64))
    for u in (um, ur):
        for y, lo, hi in ((1.03125, 1.0, 1.125), (0.25 * 2 ** -9, 0.0, 2 ** -9)):
            a, b, pos = OO.encode_levels(np.full(n, y), np.full(n // 64, 127), u, False)
            assert (a == lo).all() and (b == hi).all()
            up = np.count_nonzero(pos >= 1) / n
            assert abs(up - 0.25) < 5 * math.sqrt(0.25 * 0.75 / n)


def test_codes_round_to_themselves():
    vals = OO.CODES[np.isfinite(OO.CODES)]
    x = np.resize(np.abs(vals), 256)
    for u in (0, 65535):
        lo, _, pos = OO.encode_levels(x, np.full(4, 127), np.full(256, u), False)
        assert (lo == x).all() and (pos < 1).all()


def test_random_bits_of_steps_seeds_and_elements_are_uncorrelated():
    n = 1 << 16
    i = np.arange(n, dtype=np.uint64)
    a, b = OO.random16(3, 10, i)
    others = [OO.random16(3, 11, i), OO.random16(4, 10, i), OO.random16(3, 10, i + np.uint64(n)),
              OO.random16(3, 10, i + np.uint64(1 << 34))]
    c = lambda x, y: abs(np.corrcoef(x, y)[0, 1]) * math.sqrt(n)  # noqa: E731
    assert c(a, b) < 5
    for x, y in others:
        assert c(a, x) < 5 and c(b, y) < 5
    for d in (1, 2, 4, 64):
        assert c(a[d:], a[:-d]) < 5 and c(b[d:], b[:-d]) < 5


def test_bases_start_on_blocks():
    assert OO.bases([1, 64, 0, 65, 3]) == [0, 64, 128, 128, 256]
