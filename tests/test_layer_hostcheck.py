"""The host code of the norm, the router and the rows' way to the experts under
AddressSanitizer and UBSan (no GPU): random sizes up to the limits through the entry
points, with recording stand-ins for the launchers, every launch plan checked
(tests/hostcheck/layer_check.cpp)."""
import os

from test_hostcheck import CHECK, CSRC, ROOT, SAN, build, run


def test_layer_plans_under_sanitizers(tmp_path):
    exe = str(tmp_path / "layer_check")
    build(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "api_norm.cpp"),
           os.path.join(CSRC, "api_moe.cpp"), os.path.join(CHECK, "layer_check.cpp"), "-o", exe])
    assert ", 0 failed" in run(exe)
