"""The 8-bit product's search for a workgroup's tile: every tile of ascending offsets is found once and none twice, and
whatever the offsets hold, what is found lies within the rows.

csrc/mm_product_policy.h is plain constexpr C++, which the kernels go by; here the host C++ compiler builds it.
"""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def find(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("tiles") / "product_tile_check.so"
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dispatch_fp8_grouped_topk_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "product_tile_check.cpp"), "-o", str(out)], check=True)
    f = ctypes.CDLL(str(out)).pt_find

    def found(offset, M, m, threads, t):
        offset = np.ascontiguousarray(offset, dtype=np.int32)
        G, r = len(offset) - 1, (ctypes.c_int * 3)()
        tiles = min(M, -(-M // m) + G)
        n = f(offset.ctypes.data_as(ctypes.c_void_p), G, M, m, threads, tiles, t, r)
        return n, tuple(r)

    return found


@pytest.mark.parametrize("threads", [256, 512])
@pytest.mark.parametrize("M,G,m", [(1, 1, 16), (700, 5, 16), (1000, 300, 64), (5000, 8192, 32), (4096, 700, 256)])
def test_every_tile_of_ascending_offsets_is_found_once(find, M, G, m, threads):
    rng = np.random.default_rng(M + G)
    cut = np.sort(rng.integers(-5, M + 6, size=G + 1))                    # some of them outside: the nearest that is inside
    inside = np.clip(cut, 0, M)
    want = [(g, lo, min(m, inside[g + 1] - lo)) for g in range(G) for lo in range(inside[g], inside[g + 1], m)]
    tiles = min(M, -(-M // m) + G)
    assert len(want) <= tiles
    for t in {0, 1, len(want) // 3, len(want) // 2, len(want) - 1, len(want), tiles - 1}:
        if 0 <= t < tiles:
            n, got = find(cut, M, m, threads, t)
            assert n == (t < len(want)) and (t >= len(want) or got == want[t]), t


@pytest.mark.parametrize("threads", [256, 512])
@pytest.mark.parametrize("M", [1 << 29, (1 << 30) - 1])
def test_a_tile_of_descending_offsets_has_one_finder(find, M, threads):
    """Offsets that go up and down between 0 and M 4096 times: more than 2^32 tiles in all."""
    G, m = 8192, 256
    offset = np.zeros(G + 1, dtype=np.int64)
    offset[1::2] = M
    offset[2:G:2] = np.where(np.arange(2, G, 2) < G // 2, 0, 100)
    for t in (0, 5, (1 << 20) + 3, (1 << 21) - 1, -(-M // m) - 1, -(-M // m), -(-M // m) + G - 1):
        n, (g, m0, rows) = find(offset, M, m, threads, t)
        assert n == 1 and 0 <= g < G and 0 <= m0 and 1 <= rows <= m and m0 + rows <= M, (t, n, g, m0, rows)


def test_whatever_the_offsets_hold_what_is_found_lies_within_the_rows(find):
    rng = np.random.default_rng(3)
    for _ in range(300):
        M, G, m = int(rng.integers(1, 3000)), int(rng.integers(1, 900)), int(rng.choice([16, 32, 64, 128, 256]))
        offset = rng.integers(-2 ** 31, 2 ** 31, size=G + 1) if rng.random() < 0.3 else rng.integers(-3, M + 4, size=G + 1)
        for t in rng.integers(0, min(M, -(-M // m) + G), size=5):
            n, (g, m0, rows) = find(offset, M, m, 512, int(t))
            assert n in (0, 1)
            assert n == 0 or (0 <= g < G and 0 <= m0 and 1 <= rows <= m and m0 + rows <= M)
