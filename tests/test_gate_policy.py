"""The gate product's choice of kernel and tile, and that the GPU tests' shapes reach each one.

csrc/mm_gate_policy.h is plain constexpr C++, which the host launcher goes by; here the host C++ compiler builds it
with a small ctypes driver (tests/native/gate_policy_check.cpp).
"""
import ctypes
import os
import shutil
import subprocess

import pytest

import test_gpu_front as front

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROWS = {-1, -2}                               # dot products of rows, with one and two tokens a workgroup


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("policy") / "gate_policy_check.so"
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dispatch_fp8_grouped_topk_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "gate_policy_check.cpp"), "-o", str(out)], check=True)
    L = ctypes.CDLL(str(out))
    L.gp_variant.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    return L


@pytest.mark.parametrize("f32", [0, 1])
def test_gpu_shapes_reach_every_kernel_and_tile(lib, f32):
    tiles = set(range(lib.gp_tiles(f32)))
    reached = {}
    for T, H, E in front.GATE_TILES:
        reached.setdefault(lib.gp_variant(T, E, f32), []).append((T, H, E))
    assert set(reached) == tiles
    for v, shapes in reached.items():
        e, t = lib.gp_tile_e(f32, v), lib.gp_tile_t(f32, v)
        assert any(H == 128 for _, H, _ in shapes), (e, t)             # two steps of 64 columns
        assert any(H >= 1152 for _, H, _ in shapes), (e, t)
        assert any(T % t and E % e for T, _, E in shapes), (e, t)      # ragged both ways
    assert {lib.gp_variant(T, E, f32) for T, _, E in front.GATE_EDGES} >= ROWS


def test_gpu_shapes_of_the_float32_bits_reach_every_tile(lib):
    assert {lib.gp_variant(T, E, 1) for T, E in front.GATE_BITS} == set(range(lib.gp_tiles(1)))


@pytest.mark.parametrize("f32", [0, 1])
def test_least_bytes_a_compute_unit(lib, f32):
    """The tile's rows' bytes times the rounds of 256 workgroups, written out again."""
    for T in (1, 7, 64, 65, 128, 500, 1021, 2048, 5000, 8192, 100000, 1 << 23):
        for E in (1, 8, 33, 64, 255, 256, 1000, 8192):
            v = lib.gp_variant(T, E, f32)
            if T <= 64 and T * E <= 2048:
                assert v == (-1 if T == 1 or T * E <= 512 else -2)
                continue
            cost = [-(-(-(-E // e) * -(-T // t)) // 256) * (e * (4 if f32 else 2) + 2 * t)
                    for e, t in ((lib.gp_tile_e(f32, i), lib.gp_tile_t(f32, i)) for i in range(lib.gp_tiles(f32)))]
            assert v == cost.index(min(cost)), (T, E)
