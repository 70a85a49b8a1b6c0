"""Host-side checks of the 8-bit layer operators (no GPU): the oracle's form
against torch's e4m3 and exact arithmetic, the workspaces' sizes, and the
refusals of every entry point.  Also run under the sanitizers."""
import ctypes as C
import os
import subprocess
import sys
from fractions import Fraction

import numpy as np
import pytest

from oracle import block8_oracle as bo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
B = pytest.importorskip("zero_partitioned_mixed_buffer_amd.binding")
F32 = np.float32


@pytest.fixture(scope="module")
def L():
    return B.lib()


# ------------------------------------------------------------ the oracle's pins
@pytest.mark.parametrize("tiles", [False, True])
def test_codes_are_torchs_cast_over_the_scale(tiles):
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(3)
    x = (g.standard_normal((300, 500)) * np.exp2(g.uniform(-20, 10, (300, 1)))).astype(F32)
    codes, e = bo.encode(x, tiles)
    rows = np.repeat(e, 128, 0)[:300] if tiles else e
    y = x.astype(np.float64) / np.exp2(np.repeat(rows, 128, 1)[:, :500].astype(np.float64) - 127)
    assert np.abs(y).max() <= 448
    assert np.array_equal(codes, torch.from_numpy(y.astype(F32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    # half a step of the value, or of the smallest normal one
    err = np.abs(bo.decode(codes, e) - x)
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, np.exp2(np.repeat(rows, 128, 1)[:, :500] - 127.0) * 2.0 ** -10)).all()


def test_scale_is_the_smallest_that_fits():
    for top in (448.0, 449.0, 447.9, 224.0, 224.1, 1.0, 1e-30, 3e38, 2.0 ** -149):
        x = np.zeros((1, 128), F32)
        x[0, 77] = -top
        t = Fraction(float(abs(x[0, 77])))
        _, e = bo.encode(x)
        e = int(e[0, 0])
        fits = lambda k: t <= 448 * Fraction(2) ** (k - 127)  # noqa: E731
        assert fits(e) and (e == 1 or not fits(e - 1)) and e <= 247


def test_blocks_are_counted_from_the_first_row_and_column():
    x = np.ones((130, 257), F32)
    x[129, 256] = 1000.0
    codes, e = bo.encode(x, True)
    assert e.shape == (2, 3) and len(set(e.ravel()[:-1])) == 1 and e[1, 2] > e[0, 0]
    assert np.array_equal(bo.encode(x.T, True)[1], e.T)


# -------------------------------------------------------------- workspace sizes
def test_workspaces(L):
    ws = L.zero_block8_workspace_bytes
    assert ws(0, 5, 5) == ws(5, 0, 5) == ws(5, 5, 0) == ws(-1, 5, 5) == 0
    assert ws(1, 6400, 1600) == 0
    for m, n, k in ((768, 768, 32768), (65, 16, 8192), (300, 500, 2048), (2048, 2048, 1 << 23)):
        b = ws(m, n, k)
        assert b % 16 == 0 and (b == 0 or b >= 2 * m * n * 4), (m, n, k)
    assert ws(768, 768, 32768) > 0
    assert ws(8192, 8192, 8192) == 0
    # sizes that the product refuses
    assert ws(1 << 31, 5, 5) == ws(5, 5, (1 << 23) + 1) == ws(1 << 30, 1 << 20, 128) == 0
    nw = L.zero_rms_norm8_workspace_bytes
    assert nw(0, 100) == nw(100, 0) == nw(-1, 3) == nw(3, (1 << 23) + 1) == nw(1 << 31, 8) == 0
    for r, c in ((1, 1), (8192, 1600), (5, 1 << 23), ((1 << 31) - 1, 64)):
        assert nw(r, c) >= min(r, 64) * c * 4 and nw(r, c) % 16 == 0 and nw(r, c) <= 1 << 31


# --------------------------------------------------------------------- refusals
# Addresses that no call gets to use: far apart, aligned.
A0, A1, A2, A3, A4, A5, A6, A7 = (0x100000000000 + i * 0x1000000000 for i in range(8))


def matrix(data=A0, rows=200, cols=300, stride=None, type=B.TYPE_BF16, reserved=0):
    return B.Matrix(data, rows, cols, cols if stride is None else stride, type, reserved)


def block8(codes=A1, scales=A2, rows=200, cols=300, cs=304, ss=4, blocks=0, reserved=0):
    return B.Block8(codes, scales, rows, cols, cs, ss, blocks, reserved)


def ref(x):
    return None if x is None else C.byref(x)


BAD_MATRIX = [(dict(type=0), B.ZERO_EINVAL), (dict(type=4), B.ZERO_EINVAL), (dict(reserved=1), B.ZERO_EINVAL),
              (dict(stride=299), B.ZERO_EINVAL), (dict(data=None), B.ZERO_EINVAL), (dict(data=A0 + 1), B.ZERO_EALIGN),
              (dict(stride=1 << 62), B.ZERO_EOVERFLOW), (dict(stride=1 << 58), B.ZERO_EOVERFLOW)]
BAD_BLOCK8 = [(dict(blocks=2), B.ZERO_EINVAL), (dict(reserved=1), B.ZERO_EINVAL), (dict(cs=288), B.ZERO_EINVAL),
              (dict(ss=0), B.ZERO_EINVAL), (dict(ss=-4), B.ZERO_EINVAL), (dict(codes=None), B.ZERO_EINVAL),
              (dict(scales=None), B.ZERO_EINVAL), (dict(cs=312), B.ZERO_EALIGN), (dict(ss=6), B.ZERO_EALIGN),
              (dict(codes=A1 + 8), B.ZERO_EALIGN), (dict(scales=A2 + 2), B.ZERO_EALIGN),
              (dict(cs=(1 << 23) + 16), B.ZERO_EOVERFLOW), (dict(ss=(1 << 23) + 4), B.ZERO_EOVERFLOW)]


def test_encode_refusals(L):
    def call(x=None, rm=None, cm=None, ct=0, out=None, out_t=None):
        return L.zero_block8_encode(ref(x), rm, cm, ct, ref(out), ref(out_t), None)

    t = dict(codes=A3, scales=A4, rows=300, cols=200, cs=208, ss=4)
    assert call(None, out=block8()) == B.ZERO_EINVAL
    assert call(matrix()) == B.ZERO_EINVAL
    for bad, st in BAD_MATRIX:
        assert call(matrix(**bad), out=block8()) == st, bad
    for bad, st in BAD_BLOCK8:
        assert call(matrix(), out=block8(**bad)) == st, bad
    assert call(matrix(rows=-1), out=block8(rows=-1)) == B.ZERO_EINVAL
    assert call(matrix(rows=1 << 31), out=block8(rows=1 << 31)) == B.ZERO_EOVERFLOW
    assert call(matrix(rows=(1 << 23) + 1), out_t=block8(rows=300, cols=(1 << 23) + 1)) == B.ZERO_EOVERFLOW
    for bad in (dict(rows=199), dict(cols=301)):
        assert call(matrix(), out=block8(**bad)) == B.ZERO_EINVAL
    assert call(matrix(), out_t=block8()) == B.ZERO_EINVAL  # not the transposed size
    assert call(matrix(), out=block8(), out_t=block8(**t, blocks=1)) == B.ZERO_EINVAL
    assert call(matrix(), cm=A5, ct=0, out=block8()) == B.ZERO_EINVAL
    assert call(matrix(), cm=A5 + 1, ct=2, out=block8()) == B.ZERO_EALIGN
    assert call(matrix(), rm=A5 + 2, out=block8()) == B.ZERO_EALIGN
    # overlaps
    assert call(matrix(), out=block8(codes=A0)) == B.ZERO_EALIAS
    assert call(matrix(), out=block8(scales=A0 + 16)) == B.ZERO_EALIAS
    assert call(matrix(), out=block8(scales=A1 + 303 - 3 + 304 * 199 - 304 + 300)) == B.ZERO_EALIAS
    assert call(matrix(), rm=A1, out=block8()) == B.ZERO_EALIAS
    assert call(matrix(), cm=A2, ct=1, out=block8()) == B.ZERO_EALIAS
    assert call(matrix(), out=block8(), out_t=block8(**{**t, "codes": A1})) == B.ZERO_EALIAS
    assert call(matrix(), out=block8(), out_t=block8(**{**t, "scales": A1 + 16})) == B.ZERO_EALIAS
    # nothing to do
    assert call(matrix(rows=0, data=None), out=block8(rows=0, codes=None, scales=None)) == B.ZERO_OK


def test_norm_refusals(L):
    def call(x=None, r=None, w=A3, wt=3, eps=1e-6, h=None, y=None, rstd=A4):
        return L.zero_rms_norm8(ref(x or matrix()), ref(r), w, wt, eps, ref(h), ref(y or block8()), rstd, None)

    for bad, st in BAD_MATRIX:
        assert call(matrix(**bad)) == st, bad
        assert call(r=matrix(**{"data": A5, **bad}), h=matrix(data=A6)) in (st, B.ZERO_EINVAL), bad
        assert call(r=matrix(data=A5), h=matrix(**{"data": A6, **bad})) in (st, B.ZERO_EINVAL), bad
    for bad, st in BAD_BLOCK8:
        assert call(y=block8(**bad)) == st, bad
    assert call(y=block8(blocks=1)) == B.ZERO_EINVAL
    assert call(r=matrix(data=A5)) == call(h=matrix(data=A5)) == B.ZERO_EINVAL
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(eps=eps) == B.ZERO_EINVAL
    assert call(w=None) == call(rstd=None) == call(wt=0) == call(wt=4) == B.ZERO_EINVAL
    assert call(w=A3 + 1) == call(rstd=A4 + 2) == B.ZERO_EALIGN
    for bad in (dict(rows=199), dict(cols=299), dict(type=B.TYPE_F16)):
        assert call(r=matrix(**{"data": A5, **bad}), h=matrix(data=A6)) == B.ZERO_EINVAL
        assert call(r=matrix(data=A5), h=matrix(**{"data": A6, **bad})) == B.ZERO_EINVAL
    # h is x's memory, but not quite; the weight's; outputs over each other
    assert call(r=matrix(data=A5), h=matrix(data=A0 + 2)) == B.ZERO_EALIAS
    assert call(r=matrix(data=A5), h=matrix(data=A0, stride=301)) == B.ZERO_EALIAS
    assert call(r=matrix(data=A5), h=matrix(data=A3)) == B.ZERO_EALIAS
    assert call(y=block8(codes=A0)) == call(y=block8(scales=A3)) == call(rstd=A0) == call(rstd=A1) == B.ZERO_EALIAS
    assert call(matrix(rows=5, cols=0, data=None), y=block8(rows=5, cols=0)) == B.ZERO_EINVAL  # no mean
    assert call(matrix(rows=0, data=None), y=block8(rows=0)) == B.ZERO_OK


def test_backward_refusals(L):
    def call(dy=None, h=None, w=A3, wt=3, rstd=A4, dh=None, dx=None, dw=A6, ws=A7):
        return L.zero_rms_norm8_backward(ref(dy or matrix()), ref(h or matrix(data=A1)), w, wt, rstd, ref(dh),
                                         ref(dx or matrix(data=A2)), dw, ws, None)

    for bad, st in BAD_MATRIX:
        assert call(matrix(**bad)) == st, bad
        for name, at in (("h", A1), ("dh", A5), ("dx", A2)):
            more = {"data": at, **bad}
            if more["data"] == A0 + 1:
                more["data"] = at + 1
            assert call(**{name: matrix(**more)}) in (st, B.ZERO_EINVAL), (name, bad)
    for bad in (dict(rows=199), dict(cols=299), dict(type=B.TYPE_F32)):
        for name, at in (("h", A1), ("dh", A5), ("dx", A2)):
            assert call(**{name: matrix(**{"data": at, **bad})}) == B.ZERO_EINVAL, (name, bad)
    assert call(w=None) == call(rstd=None) == call(ws=None) == call(wt=9) == B.ZERO_EINVAL
    assert call(w=A3 + 1) == call(rstd=A4 + 1) == call(dw=A6 + 2) == call(ws=A7 + 8) == B.ZERO_EALIGN
    assert call(dx=matrix(data=A1)) == B.ZERO_EALIAS          # h is read again by nobody, but dx over it is refused
    assert call(dx=matrix(data=A0 + 2)) == B.ZERO_EALIAS      # dy, but not quite
    assert call(dw=A2) == call(dw=A0) == call(dw=A3) == B.ZERO_EALIAS
    assert call(ws=A0) == call(ws=A6) == call(ws=A2) == B.ZERO_EALIAS
    assert call(matrix(rows=0), h=matrix(rows=0), dx=matrix(rows=0), dw=None, ws=None) == B.ZERO_OK


def test_product_refusals(L):
    def call(a=None, b=None, add=None, out=None, ws=A7):
        return L.zero_block8_product(ref(a or block8()), ref(b or block8(codes=A3, scales=A4, rows=100)), ref(add),
                                     ref(out or matrix(data=A5, cols=100)), ws, None)

    for bad, st in BAD_BLOCK8:
        assert call(a=block8(**bad)) == st, bad
    for bad, st in BAD_BLOCK8:
        more = {"codes": A3, "scales": A4, "rows": 100, **bad}
        assert call(b=block8(**more)) == st, bad
    for bad, st in BAD_MATRIX:
        if "stride" in bad and bad["stride"] == 299:
            bad = dict(stride=99)
        more = {"data": A5, "cols": 100, **bad}
        if more["data"] == A0 + 1:
            more["data"] = A5 + 1
        assert call(out=matrix(**more)) == st, bad
    assert call(b=block8(codes=A3, scales=A4, rows=100, cols=301)) == B.ZERO_EINVAL
    for bad in (dict(rows=201), dict(cols=99)):
        assert call(out=matrix(**{"data": A5, "cols": 100, **bad})) == B.ZERO_EINVAL
        assert call(add=matrix(**{"data": A6, "cols": 100, **bad})) == B.ZERO_EINVAL
    assert call(add=matrix(data=A6, cols=100, type=B.TYPE_F32)) == B.ZERO_EINVAL
    for at in (A1, A2, A3, A4):
        assert call(out=matrix(data=at, cols=100)) == B.ZERO_EALIAS
    assert call(add=matrix(data=A5 + 2, cols=100)) == B.ZERO_EALIAS
    # a workspace that is needed: missing, misaligned, over an operand
    k = dict(cols=32768, cs=32768, ss=256)
    big = dict(a=block8(**k), b=block8(codes=A3, scales=A4, rows=100, **k))
    assert L.zero_block8_workspace_bytes(200, 100, 32768) > 0
    assert call(**big, ws=None) == B.ZERO_EINVAL
    assert call(**big, ws=A7 + 8) == B.ZERO_EALIGN
    for at in (A1, A2, A3, A4, A5):
        assert call(**big, ws=at) == B.ZERO_EALIAS
    # more tiles than a launch holds
    r = 1 << 30
    assert call(a=block8(rows=r), b=block8(codes=A3, scales=A4, rows=1 << 20), out=matrix(data=A5, rows=r, cols=1 << 20)) \
        == B.ZERO_EOVERFLOW
    assert call(a=block8(rows=0), out=matrix(data=A5, rows=0, cols=100)) == B.ZERO_OK


def test_columns_of_one_buffer_do_not_overlap(L):
    """Matrices of one stride side by side pass the overlap check (what fails
    then is the launch, or nothing where there is a GPU to launch on, so only
    the refusing half is called: one column more)."""
    x = matrix(cols=300, stride=1000)
    r, h = matrix(data=A0 + 600, cols=300, stride=1000), matrix(data=A0 + 1200, cols=300, stride=1000)

    def call(h):
        return L.zero_rms_norm8(ref(x), ref(r), A3, 3, -1.0, ref(h), ref(block8()), A4, None)

    assert call(h) == B.ZERO_EINVAL  # eps
    over = matrix(data=A0 + 1198, cols=300, stride=1000)
    assert L.zero_rms_norm8(ref(x), ref(r), A3, 3, 1e-6, ref(over), ref(block8()), A4, None) == B.ZERO_EALIAS


@pytest.mark.timeout(600)
def test_these_under_asan_ubsan():
    if os.environ.get("LD_PRELOAD"):
        pytest.skip("LD_PRELOAD is already set by the environment; the sanitizer runtime must come first")
    from zero_partitioned_mixed_buffer_amd import hostcheck_build
    lib = hostcheck_build.build()
    env = dict(os.environ, LD_PRELOAD=hostcheck_build.runtime(), ZERO_DP_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    env.pop("PYTEST_ADDOPTS", None)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=540)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0, out
    assert " passed" in r.stdout and "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out
