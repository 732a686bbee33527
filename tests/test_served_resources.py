"""Registers and LDS of the rotary and mixer kernels, from the compiler's kernel metadata and assembly."""
import os
import re
import shutil

import pytest

from tests.test_kernel_resources import HIPCC, _kernels
from tests.test_linattn_resources import _scratch_in_chunk_loops

pytestmark = pytest.mark.skipif(not shutil.which(HIPCC) and not os.path.exists(HIPCC), reason="no hipcc")


def test_rotary_registers(tmp_path):
    ks = {n: r for n, r in _kernels("rotary.hip", tmp_path).items() if "rotary_kernel" in n or "qknorm" in n}
    assert len(ks) == 42, sorted(ks)
    for name, r in ks.items():
        assert r["vgpr_count"] <= 168 and r.get("vgpr_spill_count", 0) == 0, (name, r)   # (three waves on a SIMD at least)


def test_mixer_registers(tmp_path):
    """Eight waves a workgroup, two on a SIMD, and a workgroup's tiles in a CU's LDS; the passes for the segments' own states
    leave room for two workgroups. No bf16 sweep spills (a load in flight that is spilled is waited for)."""
    seen = 0
    for name, r in _kernels("ssdconv.hip", tmp_path).items():
        m = re.search(r"ssdconv_sweep_kernelI([tf])Li(\d+)ELi(\d)ELb([01])ELb([01])E", name)
        if not m:
            assert r.get("vgpr_spill_count", 0) == 0, (name, r)
            continue
        seen += 1
        own = m.group(4) == "1"
        assert r["vgpr_count"] <= (128 if own else 256), (name, r)
        assert r["group_segment_fixed_size"] <= (80 if own else 160) * 1024, (name, r)
        if own or m.group(1) == "t":
            assert r.get("vgpr_spill_count", 0) == 0, (name, r)
    assert seen == 12


def test_mixer_without_spills_in_the_chunk_loop(tmp_path):
    loops = {n: k for n, k in _scratch_in_chunk_loops("ssdconv.hip", tmp_path / "ssdconv.s").items() if "sweep" in n}
    assert len(loops) == 12
    for name, n in loops.items():
        m = re.search(r"sweep_kernelI([tf])Li(\d+)ELi(\d)ELb([01])ELb([01])E", name)
        if m.group(1) == "t" or m.group(4) == "1":
            assert n == 0, (name, n)


def test_no_sweep_of_the_mixer_spills(tmp_path):
    """fp32 and bf16, whole pieces or single elements: all 24 bits of every factor in registers, and no scratch memory."""
    sweeps = {n: r for n, r in _kernels("ssdconv.hip", tmp_path).items() if "ssdconv_sweep_kernel" in n}
    assert len(sweeps) == 12
    for name, r in sweeps.items():
        assert r.get("vgpr_spill_count", 0) == 0, (name, r)
    for name, n in _scratch_in_chunk_loops("ssdconv.hip", tmp_path / "ssdconv.s").items():
        assert n == 0, (name, n)
