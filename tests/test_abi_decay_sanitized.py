"""The host code of the decayed linear attention and the state cache under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): decay_api.cpp with the rest of the C ABI, the launches replaced by stand-ins
(tests/sanitize), and tests/test_abi_decay.py run against that library in a child process."""
import os
import subprocess
import sys

import pytest


def test_decay_abi_under_sanitizers(tmp_path):
    shared = pytest.importorskip("test_abi_sanitized")  # (a tree for GPU runs may come without the sanitized builds)
    CSRC, HIPCC, ROOT, SAN = shared.CSRC, shared.HIPCC, shared.ROOT, shared.SAN
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not installed")
    rt = shared._runtime()
    if rt is None:
        pytest.skip("no AddressSanitizer runtime next to hipcc")
    stubs = os.path.join(ROOT, "tests", "sanitize")
    srcs = [os.path.join(CSRC, n) for n in ("api.cpp", "plan.cpp", "decay_api.cpp")]
    srcs += [os.path.join(stubs, n) for n in ("launch_stubs.cpp", "decay_stubs.cpp")]
    jobs, objs = [], []
    for src in srcs:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        jobs.append(subprocess.Popen([HIPCC, "-x", "hip", "--offload-host-only", "-O1", "-g", "-fPIC", "-std=c++17",
                                      "-fno-omit-frame-pointer", *SAN, "-I", os.path.join(ROOT, "include"), "-c", src,
                                      "-o", objs[-1]], stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True))
    for job in jobs:
        err = job.communicate()[1]
        assert job.returncode == 0, err[-3000:]
    lib = str(tmp_path / "libdeltarule_sanitized.so")
    r = subprocess.run([HIPCC, "-shared", "-fPIC", *SAN, *objs, "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, DELTARULE_LIBRARY=lib, LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join(ROOT, "tests", "test_abi_decay.py")], capture_output=True, text=True, env=env,
                       cwd=ROOT, timeout=600)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in out
