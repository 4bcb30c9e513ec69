"""The sizes of product_cases take the kernels named there (no GPU): the choice as the
entry points make it, with stand-ins for the launchers
(tests/hostcheck/variant_check.cpp)."""
import os
import subprocess

import pytest

from product_cases import EXPERTS, MATVEC, PRODUCTS
from test_hostcheck import CHECK, CSRC, ROOT, build


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("variants") / "variant_check")
    build(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "api_matmul.cpp"),
           os.path.join(CHECK, "variant_check.cpp"), "-o", exe])

    def ask(op, sizes):
        text = "".join(f"{op} {' '.join(map(str, s))}\n" for s in sizes)
        return subprocess.run([exe], input=text, capture_output=True, text=True, check=True,
                              timeout=60).stdout.splitlines()

    return ask


@pytest.mark.parametrize("flags", [0, 16, 64, 80])
def test_products(choice, flags):
    assert choice("mm", [(*s, flags) for s, _ in PRODUCTS]) == [w for _, w in PRODUCTS]


def test_matvec(choice):
    assert choice("mv", [s for s, _ in MATVEC]) == [w for _, w in MATVEC]


def test_experts(choice):
    assert choice("mve", [s for s, _ in EXPERTS]) == [w for _, w in EXPERTS]


def test_every_kernel_is_among_them():
    forms = {"any", "small 32 8", "small 32 4", "small 64 8", "small 64 4"}
    assert forms <= {w for _, w in PRODUCTS}
    tiles = [tuple(map(int, w.split()[1:])) for _, w in PRODUCTS if w.startswith("tile")]
    # 128 x 128, aligned and copied rows; whole tiles; parts of both sizes
    assert {(s, p) for _, _, s, p in tiles if s} == {(1, 0), (1, 1)}
    assert {n for _, n, s, _ in tiles if not s} == {1, 2, 4} and any(w and not s for w, _, s, _ in tiles)
    for cases, tokens in ((MATVEC, ["1 0", "1 1", "2 0", "2 1", "8 0", "8 1", "16 0", "16 1", "32 0", "64 0"]),
                          (EXPERTS, ["1 1", "2 1", "8 0", "16 0", "32 0", "64 0"])):
        for t in tokens:
            stages = {int(w.split()[2]) > 1 for _, w in cases if w.startswith(t + " ")}
            assert True in stages and (stages == {True, False} or t.endswith(" 1"))
