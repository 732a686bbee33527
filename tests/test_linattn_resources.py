"""Registers and LDS of the linear attention and group norm kernels, from the compiler's kernel metadata."""
import os
import re
import shutil

import pytest

from tests.test_kernel_resources import HIPCC, _kernels

pytestmark = pytest.mark.skipif(not shutil.which(HIPCC) and not os.path.exists(HIPCC), reason="no hipcc")


def test_linattn_registers(tmp_path):
    """Eight waves a workgroup, two on a SIMD: 256 VGPRs, and one workgroup's tiles in a CU's LDS.  Up to 128
    contraction columns no sweep without the decay's gradient spills (loads in flight must not be spilled: each
    spill waits for them), and no pass for the segments' states at all."""
    ks = _kernels("linattn.hip", tmp_path)
    sweeps = states = 0
    for name, r in ks.items():
        m = re.search(r"linattn_(state_)?kernelI([tf])Li(\d+)ELb([01])ELb([01])E", name)
        if not m:
            continue
        assert r["vgpr_count"] <= 256 and r["group_segment_fixed_size"] <= 160 * 1024, (name, r)
        if m.group(1):
            states += 1
            assert r.get("vgpr_spill_count", 0) == 0, (name, r)
        else:
            sweeps += 1
            if int(m.group(3)) <= 128 and m.group(4) == "0":
                assert r.get("vgpr_spill_count", 0) == 0, (name, r)
    assert sweeps == states == 24, sorted(ks)


def test_groupnorm_registers(tmp_path):
    ks = {n: r for n, r in _kernels("groupnorm.hip", tmp_path).items() if "gn_" in n}
    assert len(ks) > 20, sorted(ks)
    for name, r in ks.items():
        assert r["vgpr_count"] <= 256 and r.get("vgpr_spill_count", 0) == 0, (name, r)
