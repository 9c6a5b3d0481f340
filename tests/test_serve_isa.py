"""What the serving kernels' machine code has to hold where a GPU test cannot show it: read from the assembly that
hipcc writes for the sources (no GPU needed)."""

import os
import re
import shutil
import subprocess

import pytest

from dequant_matmul_qmv_amd import build


@pytest.fixture(scope="module")
def sample_asm(tmp_path_factory):
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("needs hipcc")
    out = str(tmp_path_factory.mktemp("isa") / "sample.s")
    cmd = [cc, *build.common_flags(), "-x", "hip", "-S", "--cuda-device-only", os.path.join(build.CSRC, "sample.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return open(out).read()


def _kernels(asm, name):
    """(mangled name, lines) of each kernel whose mangled name holds `name`."""
    for m in re.finditer(rf"^(\w*{name}\w*):.*?^\s*s_endpgm\b.*?^\.Lfunc_end", asm, re.S | re.M):
        yield m.group(1), m.group(0).splitlines()


def test_last_workgroup_sees_every_waves_stores(sample_asm):
    """sample_wide_kernel<T, true>: a workgroup counts its arrival (SamplePlan::arrived, 20 bytes in) after all of its
    waves' stores to the list and the kept weights.  A barrier does not wait for stores, so every wave has to, between
    its last store and the barrier; then one of them writes the L2 back, for the other dies, before it counts."""
    seen = 0
    for name, lines in _kernels(sample_asm, "sample_wide_kernelILi\\dELb1E"):
        seen += 1
        count = next(i for i, x in enumerate(lines) if re.search(r"global_atomic_add\b.*offset:20\b", x))
        barrier = max(i for i in range(count) if re.search(r"\bs_barrier\b", lines[i]))
        store = max(i for i in range(barrier) if re.search(r"\bglobal_store", lines[i]))
        assert re.search(r"s_waitcnt .*vmcnt\(0\)", "\n".join(lines[store:barrier])), name
        assert re.search(r"buffer_wbl2 sc1\b.*s_waitcnt .*vmcnt\(0\)", "\n".join(lines[barrier:count]), re.S), name
    assert seen == 3
