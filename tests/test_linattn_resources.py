"""Registers and LDS of the linear attention and group norm kernels, from the compiler's kernel metadata."""
import os
import re
import shutil
import subprocess

import pytest

from selective_state_space_50_amd import build_lib
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


def _scratch_in_chunk_loops(src, out):
    """{kernel: scratch accesses inside its chunk loops}: the innermost loops that hold a barrier and a matrix
    instruction, from the compiler's assembly."""
    flags = [f for f in build_lib.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([HIPCC, *flags, "--cuda-device-only", "-S", "-I", build_lib.INCLUDE, "-I", build_lib.CSRC,
                    os.path.join(build_lib.CSRC, src), "-o", str(out)], check=True, capture_output=True, timeout=600)
    res = {}
    for m in re.finditer(r"^(_ZN\w+):[^\n]*\n(.*?)^\.Lfunc_end", out.read_text(), re.M | re.S):
        lines = m.group(2).split("\n")
        at = {q.group(1): i for i, q in ((i, re.match(r"(\.LBB\w+):", s)) for i, s in enumerate(lines)) if q}
        jumps = ((i, re.match(r"\s+s_c?branch\w*\s+(\.LBB\w+)", s)) for i, s in enumerate(lines))
        loops = [(at[q.group(1)], i) for i, q in jumps if q and at[q.group(1)] <= i]
        loops = [(a, b) for a, b in loops if all(any(w in s for s in lines[a:b]) for w in ("s_barrier", "v_mfma"))]
        loops = [(a, b) for a, b in loops if not any((c, d) != (a, b) and a <= c and d <= b for c, d in loops)]
        res[m.group(1)] = sum(bool(re.match(r"\s+scratch_", s)) for a, b in loops for s in lines[a:b])
    return res


def test_sweeps_without_spills_in_the_chunk_loop(tmp_path):
    """Up to 128 contraction columns the aligned bf16 sweeps, those with the decay's gradient among them, and every
    fp32 sweep without it touch no scratch memory while they walk chunks."""
    seen = 0
    for name, n in _scratch_in_chunk_loops("linattn.hip", tmp_path / "linattn.s").items():
        m = re.search(r"linattn_kernelI([tf])Li(\d+)ELb([01])ELb([01])E", name)
        if m and int(m.group(2)) <= 128 and (m.group(3) == "0" or (m.group(1) == "t" and m.group(4) == "1")):
            seen += 1
            assert n == 0, (name, n)
    assert seen == 10
