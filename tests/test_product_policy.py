"""The 8-bit product's choice of kernel and tile, and that the GPU tests' shapes reach each one.

csrc/mm_product_policy.h is plain constexpr C++, which the host launcher goes by; here the host C++ compiler builds it
with a small ctypes driver (tests/native/product_policy_check.cpp).
"""
import ctypes
import os
import shutil
import subprocess

import pytest

import test_gpu_parts as gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("policy") / "product_policy_check.so"
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dispatch_fp8_grouped_topk_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "product_policy_check.cpp"), "-o", str(out)], check=True)
    L = ctypes.CDLL(str(out))
    L.pp_variant.argtypes = [ctypes.c_int64] * 4
    L.pp_workgroups.argtypes = [ctypes.c_int, *[ctypes.c_int64] * 3]
    L.pp_workgroups.restype = ctypes.c_int64
    return L


def test_gpu_shapes_reach_every_kernel_and_tile(lib):
    every = set(range(lib.pp_count()))
    dense = {}
    for M, N, K in gpu.DENSE:
        dense.setdefault(lib.pp_variant(M, N, K, 1), []).append((M, N, K))
    assert set(dense) == every, every - set(dense)
    for v, shapes in dense.items():
        n, m = lib.pp_n(v), lib.pp_m(v)
        assert any(M % m and N % n for M, N, _ in shapes), (n, m)          # ragged both ways
        assert any(K // 128 % 4 for _, _, K in shapes), (n, m)             # scales of a part of four blocks
        # fewer blocks than a ring holds; the second {128, 64} shares K, for long ones only
        assert v < 5 or v == 6 or any(K <= 256 for _, _, K in shapes), (n, m)
        assert any(K >= 1024 for _, _, K in shapes), (n, m)                # and more
    assert {K // 128 % 2 for _, _, K in dense[6]} == {0, 1}                # both sets of waves have a last block, or one
    grouped = {lib.pp_variant(M, N, K, G) for M, N, K, G, _ in gpu.GROUPED if G > 1}
    assert grouped == every, every - grouped


def test_no_kernel_gets_more_scales_than_its_lds_holds(lib):
    for M in (1, 7, 64, 200, 256, 300, 1000, 5000):
        for N in (8, 512, 4096, 65536):
            for K in range(128, 16385, 128):
                assert K // 128 <= lib.pp_most_blocks(lib.pp_variant(M, N, K, 1))


def test_launches_stay_within_32_bits_of_threads(lib):
    """2^23 workgroups of 512 threads, tiles and slabs that no group fills included."""
    for M, N, K, G in ((1 << 30, 8, 128, 1), (1 << 22, 8192, 128, 1), (1 << 17, 1 << 20, 128, 1), (8192, 1 << 15, 128, 8192),
                       ((1 << 30) - 1, 8, 128, 8192), (1 << 24, 2048, 2048, 64)):
        v = lib.pp_variant(M, N, K, G)
        slabs, tiles = -(-N // lib.pp_n(v)), -(-M // lib.pp_m(v)) + (G if G > 1 else 0)
        assert slabs * tiles <= 1 << 23, (M, N, K, G, v)
