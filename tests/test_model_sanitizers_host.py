"""The host code of the entry points around the verification under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/host_sanitize/model_driver.cpp with the library's sources,
host-side sanitizers on, device code unchanged."""
import os
import shutil

import pytest

from test_sanitizers_host import CLANG, HERE, HIP_HOST_SAN, ROOT, SAN, _run

SOURCES = ("capi_model", "attention", "kvcache", "probs")


def test_host_code_around_the_verification(tmp_path):
    hip = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not os.path.exists(CLANG) or not (shutil.which(hip) or os.path.exists(hip)):
        pytest.skip("ROCm compilers not present")
    objs = [str(tmp_path / (n + ".o")) for n in SOURCES]
    for n, o in zip(SOURCES, objs):
        _run([hip, "-c", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
              "-packed-fp32-ops", *HIP_HOST_SAN, "-I", os.path.join(ROOT, "include"),
              os.path.join(ROOT, "lossless_speculative_sampling_amd", "csrc", n + ".hip"), "-o", o])
    exe = str(tmp_path / "model_driver")
    _run([CLANG, "-std=c++17", "-O1", "-g", *SAN, "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
          "-D__HIP_PLATFORM_AMD__", os.path.join(HERE, "model_driver.cpp"), *objs, "-L/opt/rocm/lib", "-lamdhip64",
          "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    assert ", 0 failures" in _run([exe], env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"}, timeout=120)
