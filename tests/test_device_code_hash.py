"""The hash that keys measured figures to the built reduction kernels: other
kernels of the library do not change it, their own code does."""
import os
import re

import pytest

import ddp_bucketed_gradient_amd as D
from ddp_bucketed_gradient_amd import profiling as PF


@pytest.mark.skipif(not os.path.exists(D.HIP_LIB), reason="HIP library not built")
def test_only_the_reductions_code_counts(tmp_path):
    d = open(D.HIP_LIB, "rb").read()
    h = PF.device_code_hash()
    assert re.fullmatch("[0-9a-f]{16}", h)
    objs = PF._code_objects(PF._elf_sections(d)[b".hip_fatbin"])
    mine = [o for o in objs if b"fused_mean_kernel" in o]
    others = [o for o in objs if b"adamw_kernel" in o]
    assert len(mine) == 1 and len(others) == 1

    def with_changed_text(obj):
        text = PF._elf_sections(obj)[b".text"]
        at = d.index(obj) + obj.index(text) + len(text) // 2
        p = tmp_path / "lib.so"
        p.write_bytes(d[:at] + bytes([d[at] ^ 1]) + d[at + 1:])
        return PF.device_code_hash(str(p))
    assert with_changed_text(others[0]) == h
    assert with_changed_text(mine[0]) != h


def test_no_library_and_no_elf(tmp_path):
    assert PF.device_code_hash(str(tmp_path / "none.so")) is None
    (tmp_path / "text.so").write_text("not a library")
    assert PF.device_code_hash(str(tmp_path / "text.so")) is None
