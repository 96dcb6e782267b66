"""The argument checks of linear attention, dropout and the vocabulary's cross entropy under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU): abi.cpp is compiled with both on the host side, as in test_sanitize_cpu.py, and run with
extreme sizes (tests/sanitize/block_driver.cpp). No call may launch anything or raise a sanitizer report."""

import os
import subprocess

import pytest

from test_sanitize_cpu import CSRC, HIPCC, ROOT, SAN, _kernel_objects


@pytest.mark.slow
def test_extreme_sizes_are_refused(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not found")
    objs = _kernel_objects()
    flags = ["-O1", "-g", "-std=c++17", "-fPIC", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
             f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]
    host = []
    for src in (os.path.join(CSRC, "abi.cpp"), os.path.join(CSRC, "pack.cpp"),
                os.path.join(ROOT, "tests", "sanitize", "block_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, *flags, "-x", "c++", "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        host.append(obj)
    exe = str(tmp_path / "block_driver")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN[:4], *host, *objs, "-o", exe], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out and "LeakSanitizer" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert "0 failures" in r.stdout
