"""Host-side AddressSanitizer + UBSan run of the row operators' argument checks,
workspace sizes and plans (no GPU), built as the other operators' is
(tests/test_sanitizers_operators.py), with tests/sanitize/rows_driver.cpp.
"""
import glob
import os

import pytest

from helpers import ROOT, builder, ensure_built
from test_sanitizers import OUT, SAN_ENV, _run


def test_rows_host_code_under_asan_ubsan():
    ensure_built()
    b = builder()
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    objcopy, clangxx = (os.path.join(rocm, "llvm", "bin", n) for n in ("llvm-objcopy", "clang++"))
    if not (os.path.exists(objcopy) and os.path.exists(clangxx)):
        pytest.skip("ROCm llvm tools not found")
    out = os.path.join(OUT, "rows")
    os.makedirs(out, exist_ok=True)
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
           "-fno-sanitize-recover=all"]
    objs = []
    for src in sorted(glob.glob(os.path.join(b.CSRC, "*.hip"))):
        name = os.path.basename(src)
        if name not in ("conv2d_api.hip", "rms_norm.hip", "matmul.hip", "dropout.hip"):
            objs.append(os.path.join(b.BUILD_DIR, name + ".o"))   # as it is: not called here
            continue
        fatbin, obj = os.path.join(out, name + ".hipfb"), os.path.join(out, name + ".o")
        _run([objcopy, "--dump-section=.hip_fatbin=" + fatbin, os.path.join(b.BUILD_DIR, name + ".o")])
        _run([b.hipcc(), "--cuda-host-only", "-Xclang", "-fcuda-include-gpubinary", "-Xclang", fatbin, "-c", src,
              "-o", obj, "-O1", "-g", "-std=c++17", "-fPIC", "-I", os.path.join(ROOT, "include")] + san)
        objs.append(obj)
    drv, exe = os.path.join(out, "driver.o"), os.path.join(out, "driver")
    _run([clangxx, "-c", os.path.join(ROOT, "tests", "sanitize", "rows_driver.cpp"), "-o", drv, "-O1", "-g",
          "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
          os.path.join(rocm, "include"), "-fsanitize=address,undefined", "-fno-sanitize-recover=all"])
    _run([clangxx, "-o", exe, drv] + objs + ["-fsanitize=address,undefined", "-L", os.path.join(rocm, "lib"),
                                             "-lamdhip64", "-Wl,-rpath," + os.path.join(rocm, "lib")])
    assert "rows sanitize ok" in _run([exe], env=SAN_ENV, timeout=600)
