"""The host side of include/zq_train.h under AddressSanitizer and
UndefinedBehaviorSanitizer, with stub kernel launchers (no GPU).  The build is
also made with a planted out-of-bounds read, which must abort.  Every sanitizer
flag on a hipcc line sits behind -Xarch_host."""
from __future__ import annotations

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"
CLANGXX = "/opt/rocm/llvm/bin/clang++"


def _build(tmp_path, canary):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)):
        pytest.skip("hipcc / clang++ not installed")
    host = ["--cuda-host-only", "-O1", "-g", "-std=c++17", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
            "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all", f"-I{os.path.join(ROOT, 'include')}"]
    abi, drv, exe = (str(tmp_path / n) for n in ("abi.o", "drv.o", "driver"))
    for cmd in ([HIPCC, *host, "-c", "-o", abi,
                 os.path.join(ROOT, "weight_communication_zero_amd", "csrc", "zq_train_abi.hip")],
                [HIPCC, *host, *(["-DZQ_SANITIZER_CANARY"] if canary else []), "-c", "-o", drv, "-x", "hip",
                 os.path.join(ROOT, "tests", "sanitize", "train_abi_driver.cpp")],
                [CLANGXX, "-fsanitize=address,undefined", "-o", exe, drv, abi]):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-4000:]
    return exe


@pytest.mark.parametrize("canary", [False, True])
def test_host_validation_under_asan_and_ubsan(tmp_path, canary):
    exe = _build(tmp_path, canary)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    if canary:
        assert r.returncode != 0 and "Sanitizer" in r.stderr
    else:
        assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout + r.stderr
        assert "runtime error" not in r.stderr
