"""Helpers of the layer tests: seeded inputs in a type, and comparison with the
64-bit oracle within a derived bound."""
import numpy as np
import torch

from oracle import layers as OL

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(g, shape, t, pad=0, scale=1.0, shift=0.0):
    """A CUDA tensor of normal numbers and its values in 64 bits; with `pad` its
    rows are cut out of a wider tensor, whose rest holds NaN."""
    x = torch.from_numpy(g.normal(size=shape) * scale + shift).to(TYPES[t])
    if pad == 0:
        return x.cuda(), x.double().numpy()
    wide = torch.full(tuple(shape[:-1]) + (shape[-1] + pad,), float("nan"), dtype=TYPES[t], device="cuda")
    wide[..., :shape[-1]] = x.cuda()
    return wide[..., :shape[-1]], x.double().numpy()


def check(got, want, bound, t, what):
    """|got - want| within `bound` (fp32, first order: 1 % for the rest) and the
    rounding to type t."""
    got = got.detach().double().cpu().numpy().reshape(want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN elsewhere"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities"
    ok = ~(nan | inf)
    off = np.abs(got - want)[ok]
    room = (1.01 * bound + 1.01 * OL.rounding(np.abs(want) + bound, t))[ok]
    if (off > room).any():
        i = int(np.argmax(off - room))
        raise AssertionError(f"{what}: {int((off > room).sum())} of {off.size} off, {got[ok][i]} for {want[ok][i]}, "
                             f"room {room[i]}")


def norm_depth(cols):
    """Additions between an element and a row's sum, at most: 16 in a lane (and
    one for each 8192 columns of a long row), 6 in a wave, 16 waves."""
    return 38 + cols // 8192


def rows_depth(rows):
    """The same for a sum over rows: a lane's rows (32 workgroups at least, where
    there are that many rows), 32 rows of a workgroup, 1024 workgroups by 16ths."""
    return rows // 32 + 1 + 32 + 64 + 16
