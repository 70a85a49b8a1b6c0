"""Overlap of the 8-bit layer operators' matrices (no GPU): what the header
allows gets past the checks, what shares a byte does not.  The library's host
units are built with launchers that report "no device", so that a call that is
accepted returns ZERO_EHIP and computes nothing."""
import ctypes as C
import os
import random
import subprocess

import pytest

B = pytest.importorskip("zero_partitioned_mixed_buffer_amd.binding")
from test_block8_host import block8, matrix, ref  # noqa: E402
from zero_partitioned_mixed_buffer_amd.build_lib import CSRC, HOST_SOURCES, INCLUDE  # noqa: E402

A, FAR = 0x100000000000, 0x1000000000  # an address that no call gets to use, and others far from it
ACCEPTED = B.ZERO_EHIP


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    lib = tmp_path_factory.mktemp("nodevice") / "lib.so"
    srcs = [os.path.join(CSRC, f) for f in (*HOST_SOURCES, "zero_dp_nodevice.cpp")]
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", INCLUDE, *srcs, "-o", str(lib)], check=True)
    h = C.CDLL(str(lib))
    real = B.lib()
    for name in ("zero_block8_encode", "zero_rms_norm8", "zero_rms_norm8_backward", "zero_block8_product"):
        getattr(h, name).argtypes = getattr(real, name).argtypes
        getattr(h, name).restype = C.c_int
    return h


def norm(L, x, r, h, y=None):
    return L.zero_rms_norm8(ref(x), ref(r), A + 3 * FAR, 3, 1e-6, ref(h), ref(y or block8(A + FAR, A + 2 * FAR)),
                            A + 4 * FAR, None)


def test_columns_of_one_buffer_are_accepted(L):
    """Matrices of 300 bf16 columns in rows of 1000, side by side, in each order."""
    at = [A, A + 600, A + 1200]
    for x, r, h in ((0, 1, 2), (2, 1, 0), (1, 2, 0), (0, 2, 1)):
        m = [matrix(data=at[i], stride=1000) for i in (x, r, h)]
        assert norm(L, *m) == ACCEPTED, (x, r, h)
    x, r = matrix(data=A, stride=1000), matrix(data=A + 600, stride=1000)
    assert norm(L, x, r, matrix(data=A + 1200, stride=1000)) == ACCEPTED
    assert norm(L, x, r, matrix(data=A + 1198, stride=1000)) == B.ZERO_EALIAS   # a column too near
    assert norm(L, x, r, matrix(data=A + 1400, stride=1000)) == ACCEPTED        # up to the row's end
    assert norm(L, x, r, matrix(data=A + 1402, stride=1000)) == B.ZERO_EALIAS   # into the next row's x
    assert norm(L, x, r, x) == norm(L, x, r, r) == ACCEPTED                     # in place
    # the codes in a buffer of x's pitch
    y = block8(codes=A + 608, scales=A + 912, cs=2000, ss=2000)
    assert norm(L, x, None, None, y) == ACCEPTED
    y = block8(codes=A + 592, scales=A + 912, cs=2000, ss=2000)
    assert norm(L, x, None, None, y) == B.ZERO_EALIAS
    y = block8(codes=A + 608, scales=A + 904, cs=2000, ss=2000)
    assert norm(L, x, None, None, y) == B.ZERO_EALIAS


def bytes_of(at, rows, width, pitch):
    return {at + r * pitch + i for r in range(rows) for i in range(width)}


def test_against_every_byte(L):
    """Random small matrices of one pitch: accepted exactly where no byte of h is
    x's or residual's, or h is one of them."""
    g = random.Random(4)
    seen = {B.ZERO_EALIAS: 0, ACCEPTED: 0}
    for _ in range(20000):
        pitch, rows, cols = 2 * g.randint(8, 40), g.randint(1, 5), g.randint(1, 8)
        x, r, h = (matrix(data=A + 2 * g.randint(0, 120), rows=rows, cols=cols, stride=pitch // 2) for _ in range(3))
        if g.random() < 0.1:
            h.data = (x, r)[g.randint(0, 1)].data
        st = norm(L, x, r, h, block8(A + FAR, A + 2 * FAR, rows=rows, cols=cols, cs=16))
        sets = [bytes_of(m.data, rows, 2 * cols, pitch) for m in (x, r, h)]
        clash = any(sets[2] & s and h.data != m.data for s, m in zip(sets, (x, r)))
        if clash:
            assert st == B.ZERO_EALIAS, (pitch, rows, cols, x.data, r.data, h.data)
        elif rows > 1:
            # beside each other, or past each other's end but not yet a row apart: the latter may be refused
            apart = all(h.data == m.data or (h.data - m.data) % pitch >= 2 * cols and
                        (h.data - m.data) % pitch + 2 * cols <= pitch for m in (x, r))
            ends = all(h.data == m.data or not (min(sets[2]) <= max(s) and min(s) <= max(sets[2]))
                       for s, m in zip(sets, (x, r)))
            if apart or ends:
                assert st == ACCEPTED, (pitch, rows, cols, x.data, r.data, h.data)
        seen[st] += 1
    assert min(seen.values()) > 1000


def test_outputs_beside_inputs_are_accepted(L):
    """The other calls' outputs, in columns of an input's buffer."""
    dy, h, dx = (matrix(data=A + 600 * i, stride=1000) for i in range(3))
    assert L.zero_rms_norm8_backward(ref(dy), ref(h), A + 3 * FAR, 3, A + 4 * FAR, None, ref(dx), A + 5 * FAR,
                                     A + 6 * FAR, None) == ACCEPTED
    dx.data -= 2
    assert L.zero_rms_norm8_backward(ref(dy), ref(h), A + 3 * FAR, 3, A + 4 * FAR, None, ref(dx), A + 5 * FAR,
                                     A + 6 * FAR, None) == B.ZERO_EALIAS
    a, b = block8(), block8(A + 3 * FAR, A + 4 * FAR, rows=100)
    add, out = matrix(data=A + 5 * FAR, cols=100, stride=256), matrix(data=A + 5 * FAR + 200, cols=100, stride=256)
    assert L.zero_block8_product(ref(a), ref(b), ref(add), ref(out), None, None) == ACCEPTED
    assert L.zero_block8_product(ref(a), ref(b), ref(out), ref(add), None, None) == ACCEPTED
    assert L.zero_block8_product(ref(a), ref(b), ref(out), ref(out), None, None) == ACCEPTED
    out.data -= 2
    assert L.zero_block8_product(ref(a), ref(b), ref(add), ref(out), None, None) == B.ZERO_EALIAS
    x = matrix(data=A, stride=1000)
    t = dict(rows=300, cols=200, cs=1024)
    one, turned = block8(A + FAR, A + 2 * FAR, cs=1024), block8(A + FAR + 304, A + 3 * FAR, **t)
    assert L.zero_block8_encode(ref(x), None, None, 0, ref(one), ref(turned), None) == ACCEPTED
    turned.codes = A + FAR + 288
    assert L.zero_block8_encode(ref(x), None, None, 0, ref(one), ref(turned), None) == B.ZERO_EALIAS
