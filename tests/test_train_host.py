"""The training operators' host side (validation, workspace regions, choice of tiles, deals of tiles to
workgroups, launch bounds) under AddressSanitizer and UndefinedBehaviorSanitizer on the CPU."""
import os
import re
import shutil
import subprocess

import pytest

from test_abi import CSRC, HOSTCHECK


def test_training_host_side_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "hostcheck_train")
    srcs = [os.path.join(CSRC, f) for f in ("api_train.cpp", "train_rules.cpp", "host_rules.cpp")]
    srcs += [os.path.join(HOSTCHECK, f) for f in ("stubs.cpp", "stubs_train.cpp", "driver_train.cpp")]
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-Wall", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", *srcs, "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    env.pop("BEAM_MOE_SYNC_CHECK", None)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert res.returncode == 0, (res.stdout[-2000:], res.stderr[-4000:])
    m = re.search(r"hostcheck: (\d+) checks, 0 failed, (\d+) launches checked", res.stdout)
    assert m and int(m.group(2)) > 2000, res.stdout
