"""That every 8-bit product that fits a card can be launched, and what lies beyond is refused.

csrc/mm_product_policy.h is plain constexpr C++; here the host C++ compiler builds it with two small ctypes drivers.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

import dispatch_fp8_grouped_topk_amd as mm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MB = 1 << 20


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("launches") / "product_launch_check.so"
    native = [os.path.join(ROOT, "tests", "native", f"product_{n}_check.cpp") for n in ("policy", "launch")]
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dispatch_fp8_grouped_topk_amd", "csrc"), *native, "-o", str(out)], check=True)
    L = ctypes.CDLL(str(out))
    L.pp_variant.argtypes = [ctypes.c_int64] * 4
    L.pp_workgroups.argtypes = [ctypes.c_int, *[ctypes.c_int64] * 3]
    L.pl_items.argtypes = [ctypes.c_int, *[ctypes.c_int64] * 3, ctypes.c_int]
    L.pp_workgroups.restype = L.pl_items.restype = L.pl_groups.restype = L.pl_area.restype = ctypes.c_int64
    return L


# The last three nearly fill a card of 288 GB, with weights or with y.
SIZES = [(1, 8, 128, 1), (777, 2120, 3712, 1), (1024, 4096, 1536, 128), (65536, 4096, 7168, 256), ((1 << 30) - 1, 8, 128, 1),
         ((1 << 30) - 1, 8, 128, 8192), (4096, 1 << 20, 128, 1024), (4096, 1 << 20, 128, 2040), (1 << 20, 1 << 17, 128, 1)]


@pytest.mark.parametrize("M,N,K,G", SIZES)
def test_parts_of_a_launch_stay_within_32_bits_of_threads(lib, M, N, K, G):
    v = lib.pp_variant(M, N, K, G)
    assert lib.pl_groups() * 512 < 1 << 32 and lib.pl_groups() % 8 == 0
    items = lib.pl_items(v, M, N, G, G > 1)
    assert items < 1 << 31
    assert v == lib.pp_count() - 1 or items <= lib.pl_groups()            # the largest tile alone takes several parts
    # the items cover every tile, whatever the groups' sizes: one tile's rows are of one group
    slabs, whole = -(-N // lib.pp_n(v)), -(-M // lib.pp_m(v))
    assert items >= slabs * min(M, whole + (G if G > 1 else 0))
    assert lib.pp_workgroups(v, M, N, G) <= slabs * (whole + G)


def test_items_of_the_largest_area_fit_31_bits(lib):
    assert lib.pl_area() == 1 << 45
    for M, N in (((1 << 30) - 1, 1 << 15), (1 << 25, (1 << 20) - 8), ((1 << 25) - 1, 1 << 20)):
        for G in (1, 8192):
            for by_group in (0, 1):
                assert M * N < lib.pl_area() and lib.pl_items(lib.pp_variant(M, N, 128, G), M, N, G, by_group) < 1 << 31


def test_a_larger_area_is_refused():
    def call(M, N):
        p = mm.ProductProblem.make(M, N, 128, 1)
        return mm.library().mega_moe_block_product(ctypes.byref(p), *[i * MB + 8 for i in range(1, 5)], None, 6 * MB + 8, None)

    assert call((1 << 30) - 1, 1 << 20) == -1 and call(1 << 25, 1 << 20) == -1
    assert call((1 << 25) - 1, 1 << 20) == -3                            # misaligned: the sizes are taken
