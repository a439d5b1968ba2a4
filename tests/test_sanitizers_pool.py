"""The pool's C ABI unit with its host code under AddressSanitizer and UndefinedBehaviorSanitizer, driven by
tests/sanitize/pool_host_checks.c."""
import os
import shutil

import pytest

import test_sanitizers as base
from ssd_chunked_scan_03_amd import build

SRC = os.path.join(base.HERE, "sanitize")


def test_pool_host_code_under_address_and_undefined_sanitizers(tmp_path):
    hipcc = build.HIPCC
    if not (os.path.exists(hipcc) or shutil.which(hipcc)):
        pytest.skip("hipcc not available")
    hsan = [a for f in base.SAN for a in ("-Xarch_host", f)]  # host code only
    abi, stubs, drv, exe = (tmp_path / n for n in ("abi.o", "stubs.o", "checks.o", "checks"))
    base._run([hipcc, f"--offload-arch={build.ARCH}", "-O1", "-g", "-std=c++17", "-fPIC", *hsan,
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-c", os.path.join(build.CSRC, "pool_abi.hip"), "-o", str(abi)])
    base._run(["g++", "-O1", "-g", "-std=c++17", *base.SAN, "-c", os.path.join(SRC, "pool_launch_stubs.cpp"), "-o", str(stubs)])
    base._run(["gcc", "-O1", "-g", "-std=c11", *base.SAN, f"-I{build.INCLUDE}", "-c",
               os.path.join(SRC, "pool_host_checks.c"), "-o", str(drv)])
    base._run([hipcc, f"--offload-arch={build.ARCH}", *hsan, str(drv), str(abi), str(stubs), "-o", str(exe)])
    r = base._run([str(exe)], env=base.ENV, timeout=300)
    assert r.stdout.strip().endswith("OK"), r.stdout
