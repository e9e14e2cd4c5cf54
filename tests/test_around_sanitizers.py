"""The validation and workspace sizing of the operators around the recurrence
under AddressSanitizer and UndefinedBehaviorSanitizer (host code only), driven
by tests/sanitize/around_driver.c with 700,000 argument sets."""
import glob
import os
import shutil

import pytest

from test_sanitizers import CSRC, ENV, HERE, ROCM, ROOT, SAN, _run


@pytest.mark.timeout(900)
def test_around_validation_under_asan_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or os.path.join(ROCM, "bin", "hipcc")
    clang = os.path.join(ROCM, "llvm", "bin", "clang")
    if not (os.path.exists(hipcc) and os.path.exists(clang)):
        pytest.skip("the ROCm toolchain is needed for the host-only library build")
    host_san = []
    for f in SAN:                       # host side only: no sanitizer in device code
        host_san += ["-Xarch_host", f]
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + [os.path.join(CSRC, "pdn_api.cpp")]

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([hipcc, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, *host_san, "-c", src, "-o", obj])
        return obj

    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(max_workers=min(len(srcs), 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    lib = str(tmp_path / "libpdn_san.so")
    _run([hipcc, "-shared", "-fPIC", "--offload-arch=gfx950", *host_san, *objs, "-o", lib])
    exe = str(tmp_path / "around_driver")
    _run([clang, "-O1", "-g", "-std=c11", *SAN, os.path.join(HERE, "around_driver.c"),
          "-I" + os.path.join(ROOT, "include"), lib, "-Wl,-rpath," + str(tmp_path),
          "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", exe])
    r = _run([exe], env=ENV, timeout=300)
    assert " 0 inconsistent answers" in r.stdout, r.stdout
    assert int(r.stdout.split(" sets, ")[1].split(" accepted")[0]) > 100000, r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
    print(r.stdout)
