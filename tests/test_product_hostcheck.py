"""The products' host code under AddressSanitizer and UBSan (no GPU): random
sizes up to the limits through the entry points of csrc/api_matmul.cpp, with
recording stand-ins for the launchers, every launch plan checked
(tests/hostcheck/product_check.cpp)."""
import os

from test_hostcheck import CHECK, CSRC, ROOT, SAN, build, run


def test_product_plans_under_sanitizers(tmp_path):
    exe = str(tmp_path / "product_check")
    build(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "api_matmul.cpp"),
           os.path.join(CHECK, "product_check.cpp"), "-o", exe])
    assert ", 0 failed" in run(exe)
