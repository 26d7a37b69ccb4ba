"""The order that verify_pick_kernel's last workgroup relies on, in the code that is
built from decode_verify.hip: a part's sums are stored past the die's caches
(sc1) and waited for before the count of finished parts is added to."""
import os
import re
import shutil
import subprocess

import pytest

from scale_invariant_row_amd import build as builder


def test_sums_are_stored_before_they_are_counted(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("needs hipcc")
    out = tmp_path / "verify.s"
    r = subprocess.run([hipcc, *builder.CFLAGS, "-Wno-unused-command-line-argument", "-S", "--cuda-device-only",
                        os.path.join(builder.CSRC, "decode_verify.hip"),
                        "-o", str(out)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    kernels = re.findall(r"^(_ZN3dsr18verify_pick_kernel\w+):[^\n]*\n(.*?)^\.Lfunc_end", out.read_text(), re.M | re.S)
    assert len(kernels) == 2
    for name, code in kernels:
        lines = [line.strip() for line in code.splitlines()]
        adds = [i for i, line in enumerate(lines) if line.startswith("global_atomic_add")]
        stores = [i for i, line in enumerate(lines) if line.startswith("global_store_dwordx2") and "sc1" in line]
        assert len(adds) == 1 and len(stores) == 2 and max(stores) < adds[0], name
        assert "s_waitcnt vmcnt(0)" in lines[max(stores):adds[0]], name
