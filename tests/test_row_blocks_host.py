"""The tiles that the grouped and gated products find on the device from their offsets, with what each reaches, run
on the CPU lane by lane (UndefinedBehaviorSanitizer)."""
import os
import re
import shutil
import subprocess

import pytest

from test_abi import CSRC, HOSTCHECK


def test_row_blocks_on_the_cpu(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "hostcheck_rows")
    srcs = [os.path.join(HOSTCHECK, "driver_rows.cpp"), os.path.join(CSRC, "step_rules.cpp"), os.path.join(CSRC, "train_rules.cpp")]
    cmd = [gxx, "-std=c++17", "-O2", "-g", "-Wall", "-Wno-unused-function", "-Wno-unknown-pragmas", "-fsanitize=undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", *srcs, "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-4000:]
    res = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, (res.stdout[-2000:], res.stderr[-4000:])
    m = re.search(r"hostcheck: (\d+) checks, 0 failed", res.stdout)
    assert m and int(m.group(1)) > 1000000, res.stdout
