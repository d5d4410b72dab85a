"""The random bits of the 8-bit AdamW states, from the functions that the kernel
shares with the host, against the oracle's: tiles at the start, at odd places
and around group 2^32, where the index's low word wraps."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import optim as OO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = tmp_path_factory.mktemp("bits") / "optim_bits"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror",
                    os.path.join(ROOT, "tests", "c", "optim_bits.cpp"), "-o", str(exe)], check=True)
    return str(exe)


W = 1 << 32


@pytest.mark.parametrize("seed,t", [(0, 1), (12345678901234567890, 1000003)])
@pytest.mark.parametrize("tile", [0, 16, W - 1024, W - 1024 + 16, W - 528, W - 16, W, W + 16, 5 * W - 272, 7 * W])
def test_bits_of_a_tile(program, seed, t, tile):
    index = np.uint64(4 * tile) + np.arange(4096, dtype=np.uint64)
    m, r = OO.random16(seed, t, index)
    for threads in (64, 256):
        out = subprocess.run([program, str(seed), str(t), str(tile), str(threads)], capture_output=True, text=True,
                             check=True, timeout=60).stdout
        x = np.array([[int(y) for y in line.split()] for line in out.splitlines()])
        assert np.array_equal(x[:, 0], np.arange(4096))
        assert np.array_equal(x[:, 1] >> 16, m) and np.array_equal(x[:, 1] & 0xFFFF, r)
