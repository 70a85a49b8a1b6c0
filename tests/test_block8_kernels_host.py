"""The choice of the 8-bit product's kernel (no GPU): the tested sizes go to the
kernels that they are meant for, and launches stay within their limits over the
whole range of sizes.  The library's own header is compiled for the host."""
import ctypes as C
import os
import random
import subprocess

import pytest

import block8_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_partitioned_mixed_buffer_amd", "csrc")
SOURCE = """
#include "zero_dp_block8.h"
extern "C" {
int shape(int64_t m, int64_t n, int64_t k, int exact) { return zdp::product_shape(m, n, k, exact != 0); }
int64_t tiles(int64_t m, int64_t n) { return zdp::product_tiles(m, n); }
int64_t rest(int64_t m, int64_t n) { return zdp::product_rest(zdp::product_tiles(m, n)); }
int parts(int64_t m, int64_t n, int64_t k) { return zdp::product_parts(m, n, k); }
int64_t few_groups(int64_t stream, int64_t other) { return zdp::product_few_groups(stream, other); }
}
"""


@pytest.fixture(scope="module")
def H(tmp_path_factory):
    at = tmp_path_factory.mktemp("choice")
    src, lib = at / "choice.cpp", at / "choice.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(lib)], check=True)
    h = C.CDLL(str(lib))
    i64 = C.c_int64
    h.shape.argtypes, h.tiles.argtypes, h.rest.argtypes = [i64, i64, i64, C.c_int], [i64, i64], [i64, i64]
    h.parts.argtypes, h.few_groups.argtypes = [i64, i64, i64], [i64, i64]
    for f in (h.tiles, h.rest, h.few_groups):
        f.restype = i64
    return h


@pytest.mark.parametrize("case", cases.PRODUCTS + cases.MASKED + cases.EMPTY + cases.FAR)
def test_tested_sizes_reach_their_kernels(H, case):
    kernel, quarters, parts, m, n, k = case
    for exact in (0, 1):
        assert H.shape(m, n, k, exact) == kernel
    assert (kernel == cases.LARGE and H.rest(m, n) > 0) == quarters
    assert H.parts(m, n, k) == parts


def test_every_kernel_has_sizes():
    for group in (cases.PRODUCTS,):
        assert {c[0] for c in group} == {cases.FEW_B, cases.FEW_A, cases.SMALL, cases.MEDIUM, cases.LARGE}
    for group in (cases.MASKED, cases.EMPTY, cases.FAR):
        assert {c[0] for c in group} == {cases.SMALL, cases.MEDIUM, cases.LARGE}
    assert any(c[0] == cases.LARGE and not c[1] for c in cases.PRODUCTS)


# us in small, medium and large tiles, an MI355X: (fp32 out, m, n, k)
MEASURED = {
    (0, 2048, 4800, 1600): (30.3, 27.0, 26.4), (0, 4096, 2304, 768): (18.5, 14.5, 14.2),
    (0, 4096, 4800, 768): (32.6, 28.1, 30.3), (0, 8192, 768, 768): (13.5, 14.3, 12.8),
    (0, 8192, 1600, 4096): (73.8, 73.1, 52.4), (0, 8192, 4800, 4096): (217.4, 159.5, 167.0),
    (0, 5333, 3500, 768): (35.0, 28.8, 31.2), (0, 6400, 6400, 768): (56.8, 49.4, 46.3),
    (0, 11000, 2000, 1600): (60.3, 44.7, 49.9), (1, 2900, 2900, 4096): (98.7, 73.8, 84.0),
    (1, 4096, 4800, 768): (49.9, 42.4, 43.7), (1, 8192, 768, 4096): (64.1, 63.9, 76.2),
    (1, 8192, 4800, 768): (110.1, 83.0, 86.2), (1, 8192, 4800, 4096): (348.4, 302.0, 294.0),
    (1, 16384, 1600, 768): (72.3, 62.0, 57.3), (1, 16384, 1600, 4096): (245.2, 226.9, 196.4),
    (1, 6400, 6400, 1600): (165.0, 139.8, 132.3), (1, 11000, 2000, 768): (59.6, 45.5, 51.2),
}


@pytest.mark.parametrize("at", MEASURED)
def test_choice_of_tiles_is_near_the_fastest(H, at):
    exact, m, n, k = at
    us = MEASURED[at]
    assert us[H.shape(m, n, k, exact) - cases.SMALL] <= 1.09 * min(us)


def test_launches_stay_within_their_limits(H):
    """Random sizes over the whole range: fewer than 2^32 lanes to a launch (and
    65536 groups along its second axis), parts for small tiles alone, none of
    them empty, and as many quarters as there are CUs at most."""
    g = random.Random(1)
    size = {cases.SMALL: (128, 128, 256), cases.MEDIUM: (192, 256, 512), cases.LARGE: (256, 256, 512)}
    seen = set()
    for _ in range(200000):
        m, n = (int(2 ** g.uniform(0, 30.99)) for _ in range(2))
        k = int(2 ** g.uniform(0, 23))
        if H.tiles(m, n) > 1 << 22:
            continue
        for exact in (0, 1):
            shape, parts = H.shape(m, n, k, exact), H.parts(m, n, k)
            seen.add(shape)
            if shape in size:
                bm, bn, threads = size[shape]
                tiles = -(-m // bm) * -(-n // bn)
                assert tiles * threads * parts < 1 << 32, (m, n, k)
                assert parts == 1 or (shape == cases.SMALL and tiles * parts <= 256)
                blocks = -(-k // 128)
                per = (-(-blocks // parts) + 3) // 4 * 4
                assert (parts - 1) * per < blocks and 0 <= H.rest(m, n) <= 64
            else:
                stream, other = (n, m) if shape == cases.FEW_B else (m, n)
                assert parts == 1 and H.few_groups(stream, other) <= 1024
    assert seen == {cases.FEW_B, cases.FEW_A, cases.SMALL, cases.MEDIUM, cases.LARGE}
