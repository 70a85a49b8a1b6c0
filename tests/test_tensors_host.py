"""Host-side checks of the tensor-list operators (no GPU): the oracle's 8-bit
form against torch's e4m3 and exact arithmetic, the list's plan, and the
refusals of every entry point.  Also run under the sanitizers."""
import ctypes as C
import os
import subprocess
import sys
from fractions import Fraction

import numpy as np
import pytest

from oracle import tensor_oracle as to

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
B = pytest.importorskip("zero_partitioned_mixed_buffer_amd.binding")
F32 = np.float32


@pytest.fixture(scope="module")
def L():
    return B.lib()


# ------------------------------------------------------------ the oracle's pins
def test_code_values_are_torchs():
    torch = pytest.importorskip("torch")
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(to.code_values(), want, equal_nan=True)
    assert np.nanmax(to.code_values()) == 448.0


@pytest.mark.parametrize("root", [False, True])
def test_nearest_is_torchs_cast(root):
    """Nearest rounding over the block's scale equals torch's cast."""
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(3)
    x = (g.standard_normal(32 * 400) * np.exp2(g.uniform(-20, 10, 32 * 400))).astype(F32)
    x = np.abs(x) if root else x
    codes, e = to.mx8_encode(x, root)
    y = (np.sqrt(x) if root else x).reshape(-1, 32).astype(np.float64) / np.exp2(e - 127.0)[:, None]
    assert np.abs(y).max() <= 448 and (np.abs(y).max(axis=1) > 224).all()
    want = torch.from_numpy(y.astype(F32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(-1)
    if root:
        want = np.where((want == 0) & (x > 0), 1, want)
    assert np.array_equal(codes, want)


def test_stochastic_rounding_is_exact_in_its_probability():
    """Over all 2^20 random parts an element rounds up exactly as often as
    the part that is cut off says (counted in steps of 2^-20)."""
    r = np.arange(1 << 20, dtype=np.uint64)
    vals = to.code_values()
    for top, x in ((448.0, 3.3), (448.0, 0.01), (300.0, -17.77), (2.0 ** -100, 1.7e-31)):
        x32 = F32(x)
        blk = np.full((1, 32), x32, F32)
        blk[0, 31] = F32(top)
        _, e = to.mx8_encode(blk.reshape(-1))
        y = Fraction(abs(float(x32))) / Fraction(2) ** (int(e[0]) - 127)
        step = Fraction(2) ** (max(int(np.floor(np.log2(float(y)))), -6) - 3)
        frac = y / step - (y / step).__floor__()
        many = np.full((1 << 15, 32), x32, F32)
        many[:, 31] = F32(top)
        up = 0
        for part in range(32):  # a block's first element meets every random part once
            words = np.zeros((1 << 15, 32), np.uint64)
            words[:, 0] = r[part << 15:(part + 1) << 15] << np.uint64(12)
            codes, _ = to.mx8_encode(many.reshape(-1), words=words.reshape(-1))
            got = np.abs(vals[codes.reshape(-1, 32)[:, 0]])
            low = float((y / step).__floor__() * step)
            assert np.isin(got, (low, low + float(step))).all()
            up += int((got > low).sum())
        # floor(y/step + R/2^20) is up iff R >= 2^20 (1 - frac)
        assert up == (1 << 20) - -((-(1 << 20) * (1 - frac)).__floor__())


def test_random_words_are_even():
    """Words of neighbouring elements, steps and seeds: every bit is set half
    the time (n = 2^16 words: standard deviation 2^-9, six of them allowed),
    and neighbouring words share half their bits."""
    n = 1 << 16
    sets = [to.random_words(n, 0, 1), to.random_words(n, 0, 2), to.random_words(n, 1, 1),
            to.random_words(n, 1 << 32, 1), to.random_words(n, 0, 1, 1 << 31)]
    bits = [((s[:, None] >> np.arange(32, dtype=np.uint64)) & np.uint64(1)).astype(float) for s in sets]
    tol = 6 * 2.0 ** -9
    for b in bits:
        assert np.abs(b.mean(axis=0) - 0.5).max() < tol
        assert np.abs((b[1:] != b[:-1]).mean(axis=0) - 0.5).max() < tol
    for i in range(len(bits)):
        for j in range(i):
            assert np.abs((bits[i] != bits[j]).mean(axis=0) - 0.5).max() < tol
    m, r = sets[0] >> np.uint64(12), (sets[0] & np.uint64(0xFFFF)) << np.uint64(4)
    assert abs(np.corrcoef(m.astype(float), r.astype(float))[0, 1]) < 6 / np.sqrt(n)


def test_stochastic_variance_follows_and_nearest_does_not():
    """What the rounding mode is for: gradients whose size drops to a third.
    The exact variance falls to about a ninth in 8000 steps; stochastic
    8-bit states follow it, nearest ones stay."""
    g = np.random.default_rng(5)
    n = 32 * 8
    kinds = {"exact": None, "stochastic": to.TensorAdam([np.zeros(n)], 8, lr=0.0),
             "nearest": to.TensorAdam([np.zeros(n)], 8, lr=0.0, stochastic=False)}
    start = np.full(n, 1e-6, F32)
    for k in ("stochastic", "nearest"):
        kinds[k].v = [to.mx8_encode(start, True)]
    exact = start.astype(np.float64)
    for t in range(4000):
        x = (g.standard_normal(n) * 3e-4).astype(F32)
        x[::32] = 1e-3  # the block's largest stays, so its scale does too
        exact = 0.999 * exact + 0.001 * x.astype(np.float64) ** 2
        for k in ("stochastic", "nearest"):
            kinds[k].step([x])
    rest = np.arange(n) % 32 != 0
    sr = to.mx8_decode(*kinds["stochastic"].v[0], root=True)[rest].astype(np.float64)
    rn = to.mx8_decode(*kinds["nearest"].v[0], root=True)[rest].astype(np.float64)
    want = exact[rest].mean()
    assert abs(sr.mean() / want - 1) < 0.25 and rn.mean() > 5 * want


# ------------------------------------------------------------------------ plan
def _tensors(n, count=1, base=1 << 20, gap=1 << 16, mx=False, param=True):
    """Descriptors over made-up device addresses."""
    arr = (B.Tensor * max(count, 1))()
    at = base
    for i in range(count):
        for k in ("master", "grad", "exp_avg", "exp_avg_sq") + (("param",) if param else ()) + \
                (("avg_scale", "sq_scale") if mx else ()):
            setattr(arr[i], k, at)
            at += gap
        arr[i].n = n[i] if isinstance(n, (list, tuple)) else n
    return arr


def _plan(L, arr, count, g=2, p=2, s=1, cap=None):
    info = B.TensorListInfo()
    st = L.zero_tensors_plan(arr, count, g, p, s, C.byref(info), None, 0)
    if st != B.ZERO_ECAPACITY:
        return st, info, None
    size = int(info.table_bytes) if cap is None else cap
    buf = C.create_string_buffer(size + 16)
    at = (C.addressof(buf) + 15) // 16 * 16
    st = L.zero_tensors_plan(arr, count, g, p, s, C.byref(info), at, size)
    return st, info, C.string_at(at, size)


def test_plan_table(L):
    n = [0, 1, 4096, 4097, 0, 12289]
    arr = _tensors(n, 6)
    arr[5].flat_off = 2 ** 40
    st, info, raw = _plan(L, arr, 6)
    assert st == B.ZERO_OK
    assert (info.n_tensors, info.grad_type, info.param_type, info.state_type) == (6, 2, 2, 1)
    assert info.n_elems == sum(n) and info.n_chunks == 1 + 1 + 2 + 4
    desc = np.frombuffer(raw[:6 * 80], dtype=np.uint64).reshape(6, 10)
    for i in range(6):
        assert list(desc[i][:5]) == [arr[i].master, arr[i].grad, arr[i].param, arr[i].exp_avg, arr[i].exp_avg_sq]
        assert desc[i][7] == n[i] and desc[i][8] == arr[i].flat_off
    ref = np.frombuffer(raw[6 * 80:6 * 80 + 8 * info.n_chunks], dtype=np.int32).reshape(-1, 2)
    assert ref.tolist() == [[1, 0], [2, 0], [3, 0], [3, 1], [5, 0], [5, 1], [5, 2], [5, 3]]


def test_plan_empty_list(L):
    st, info, _ = _plan(L, None, 0)
    assert st == B.ZERO_OK and info.n_chunks == 0 and info.table_bytes == 0


def test_plan_refusals(L):
    ok = _tensors(100)
    info = B.TensorListInfo()
    for g, p, s in ((0, 2, 1), (4, 2, 1), (2, 1, 1), (2, 4, 1), (2, 2, 2), (2, 2, 5), (2, 2, 0)):
        assert L.zero_tensors_plan(ok, 1, g, p, s, C.byref(info), None, 0) == B.ZERO_EINVAL, (g, p, s)
    assert L.zero_tensors_plan(ok, 1, 2, 2, 1, None, None, 0) == B.ZERO_EINVAL
    assert L.zero_tensors_plan(None, 1, 2, 2, 1, C.byref(info), None, 0) == B.ZERO_EINVAL
    assert L.zero_tensors_plan(ok, -1, 2, 2, 1, C.byref(info), None, 0) == B.ZERO_EINVAL
    assert L.zero_tensors_plan(ok, 1, 2, 2, 1, C.byref(info), None, 8) == B.ZERO_EINVAL
    assert _plan(L, ok, 1, cap=16)[0] == B.ZERO_ECAPACITY
    for field in ("master", "grad", "param", "exp_avg", "exp_avg_sq"):
        arr = _tensors(100)
        setattr(arr[0], field, None)
        assert _plan(L, arr, 1)[0] == B.ZERO_EINVAL, field
    for field in ("avg_scale", "sq_scale"):
        arr = _tensors(100, mx=True)
        assert _plan(L, arr, 1, s=4)[0] == B.ZERO_OK
        assert _plan(L, arr, 1, s=1)[0] == B.ZERO_EINVAL
        setattr(arr[0], field, None)
        assert _plan(L, arr, 1, s=4)[0] == B.ZERO_EINVAL
    assert _plan(L, ok, 1, p=0)[0] == B.ZERO_EINVAL  # a copy that no type names
    for field, off, want in (("master", 2, -2), ("grad", 1, -2), ("param", 1, -2), ("exp_avg", 2, -2),
                             ("exp_avg_sq", 1, -2), ("grad", 2, 0), ("master", 4, 0), ("param", 2, 0)):
        arr = _tensors(100)
        setattr(arr[0], field, getattr(arr[0], field) + off)
        assert _plan(L, arr, 1)[0] == want, (field, off)
    arr = _tensors(100)
    arr[0].n = -1
    assert _plan(L, arr, 1)[0] == B.ZERO_EINVAL
    arr[0].n = 2 ** 62
    assert _plan(L, arr, 1)[0] == B.ZERO_EOVERFLOW
    arr[0].n, arr[0].flat_off = 100, 2 ** 63 - 50
    assert _plan(L, arr, 1)[0] == B.ZERO_EOVERFLOW
    arr[0].flat_off = -1
    assert _plan(L, arr, 1)[0] == B.ZERO_EINVAL
    arr[0].flat_off, arr[0].reserved = 0, 1
    assert _plan(L, arr, 1)[0] == B.ZERO_EINVAL


def test_plan_overlaps(L):
    """The same tensor twice, neighbours that touch or overlap by a byte, and
    gradients that may be shared."""
    twice = _tensors(64, 2)
    C.memmove(C.addressof(twice[1]), C.addressof(twice[0]), C.sizeof(B.Tensor))
    assert _plan(L, twice, 2)[0] == B.ZERO_EALIAS
    fields = ("master", "param", "exp_avg", "exp_avg_sq", "avg_scale", "sq_scale")
    size = {"master": 4, "param": 2, "exp_avg": 1, "exp_avg_sq": 1, "avg_scale": 1 / 32, "sq_scale": 1 / 32}
    for f in fields:
        for other in fields + ("grad",):
            if f == other:
                continue
            arr = _tensors(64, 2, mx=True)
            end = getattr(arr[1], f) + int(64 * size[f])
            setattr(arr[0], other, end)
            if other not in ("master", "param", "grad") or end % 4 == 0:
                assert _plan(L, arr, 2, s=4)[0] == B.ZERO_OK, (f, other)
            arr = _tensors(64, 2, mx=True)
            setattr(arr[0], other, getattr(arr[1], f))
            assert _plan(L, arr, 2, s=4)[0] == B.ZERO_EALIAS, (f, other)
    arr = _tensors(64, 2)
    arr[1].grad = arr[0].grad
    assert _plan(L, arr, 2)[0] == B.ZERO_OK
    assert _plan(L, twice, 2, p=0, s=0)[0] == B.ZERO_OK  # a norm of the same gradient twice


def test_plan_gradients_alone(L):
    arr = (B.Tensor * 2)()
    for i in range(2):
        arr[i].grad, arr[i].n = (i + 1) << 20, 5000
    st, info, _ = _plan(L, arr, 2, p=0, s=0)
    assert st == B.ZERO_OK and info.n_chunks == 4


# ----------------------------------------------------------------- async calls
def _hp(**kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    d.update(kw)
    return B.adam_hp(**d)


def _step(L, info, hp=None, table=1 << 30, scale=1.0, ctl=1 << 32, ovf=1 << 33, sq=1 << 34, rounding=0, seed=0,
          ws=1 << 35):
    return L.zero_tensors_adam_step(C.byref(info), table, C.byref(hp or _hp()), scale, ctl, ovf, sq, rounding, seed,
                                    ws, None)


def test_step_refusals(L):
    """Every refusal comes before a launch (nothing here reaches a device)."""
    _, info, _ = _plan(L, _tensors(100), 1)
    _, mx, _ = _plan(L, _tensors(100, mx=True), 1, s=4)
    _, norm, _ = _plan(L, _tensors(100), 1, p=0, s=0)
    E = B.ZERO_EINVAL
    assert _step(L, norm) == E
    for kw in (dict(table=None), dict(ctl=None), dict(ws=None), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-320), dict(rounding=1),
               dict(rounding=2)):
        assert _step(L, info, **kw) == E, kw
    assert _step(L, mx, rounding=2) == E
    for kw in (dict(table=(1 << 30) + 8), dict(ctl=(1 << 32) + 4), dict(ovf=(1 << 33) + 2), dict(sq=(1 << 34) + 4),
               dict(ws=(1 << 35) + 8)):
        assert _step(L, info, **kw) == B.ZERO_EALIGN, kw
    for kw in (dict(ovf=1 << 32), dict(sq=1 << 35), dict(ctl=1 << 30), dict(ws=1 << 30)):
        assert _step(L, info, **kw) == B.ZERO_EALIAS, kw
    nan = float("nan")
    for bad in (dict(lr=-1.0), dict(lr=nan), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(weight_decay=-1),
                dict(max_grad_norm=-1.0), dict(max_grad_norm=nan), dict(scale_interval=-1),
                dict(scale_interval=1, scale_growth=0.0), dict(scale_interval=1, scale_backoff=nan)):
        assert _step(L, info, _hp(**bad)) == E, bad
    assert _step(L, info, _hp(max_grad_norm=1.0), sq=None) == E
    assert _step(L, info, _hp(max_grad_norm=1.0), ovf=None) == E
    assert _step(L, info, _hp(scale_interval=5), ovf=None) == E
    for f, v in (("n_tensors", -1), ("n_chunks", -1), ("grad_type", 0), ("param_type", 1), ("state_type", 7),
                 ("reserved", 1), ("n_elems", -1), ("table_bytes", -1)):
        bad = B.TensorListInfo.from_buffer_copy(info)
        setattr(bad, f, v)
        assert _step(L, bad) == E, f


def test_norm_refusals(L):
    _, info, _ = _plan(L, _tensors(100), 1, p=0, s=0)

    def call(table=1 << 30, scale=1.0, ctl=None, ovf=1 << 33, sq=1 << 34, ws=1 << 35):
        return L.zero_tensors_grad_norm(C.byref(info), table, scale, ctl, ovf, sq, ws, None)

    for kw in (dict(table=None), dict(ovf=None), dict(sq=None), dict(ws=None), dict(scale=0.0), dict(scale=1e-320)):
        assert call(**kw) == B.ZERO_EINVAL, kw
    for kw in (dict(ovf=(1 << 33) + 1), dict(sq=(1 << 34) + 4), dict(ws=(1 << 35) + 8), dict(ctl=(1 << 32) + 4)):
        assert call(**kw) == B.ZERO_EALIGN, kw
    for kw in (dict(ovf=1 << 34), dict(sq=1 << 30), dict(ctl=1 << 33), dict(ws=1 << 30)):
        assert call(**kw) == B.ZERO_EALIAS, kw


def test_mx8_refusals(L):
    def enc(x=1 << 30, n=100, root=0, c=1 << 31, s=1 << 32, rounding=0, step=0, off=0):
        return L.zero_mx8_encode(x, n, root, c, s, rounding, 0, step, off, None)

    def dec(x=1 << 30, n=100, root=0, c=1 << 31, s=1 << 32):
        return L.zero_mx8_decode(c, s, n, root, x, None)

    for f in (enc, dec):
        for kw in (dict(x=None), dict(c=None), dict(s=None), dict(n=-1), dict(root=2)):
            assert f(**kw) == B.ZERO_EINVAL, kw
        assert f(x=(1 << 30) + 2) == B.ZERO_EALIGN
        assert f(n=2 ** 62) == B.ZERO_EOVERFLOW
        for kw in (dict(c=(1 << 30) + 399), dict(s=(1 << 31) + 99), dict(s=(1 << 30) - 3)):
            assert f(**kw) == B.ZERO_EALIAS, kw
        assert f(n=0, x=None, c=None, s=None) == B.ZERO_OK
    assert enc(rounding=2) == enc(step=-1) == enc(off=-1) == B.ZERO_EINVAL
    assert enc(off=2 ** 63 - 50) == B.ZERO_EOVERFLOW


def test_python_refusals():
    """The binding's own checks, on host tensors (a list's tensors have to be
    device tensors of the current device)."""
    torch = pytest.importorskip("torch")
    from zero_partitioned_mixed_buffer_amd import TensorAdam
    g, m = [torch.zeros(4, dtype=torch.float16)], [torch.zeros(4)]
    with pytest.raises(ValueError, match="device tensor"):
        B.tensor_list(g)
    with pytest.raises(ValueError, match="torch tensors"):
        B.tensor_list([None])
    with pytest.raises(ValueError, match="come together"):
        B.tensor_list(g, m)
    with pytest.raises(ValueError, match="gradients alone"):
        B.tensor_list(g, params=g)
    with pytest.raises(ValueError, match="entries"):
        B.tensor_list(g, m * 2, exp_avg=m, exp_avg_sq=m)
    with pytest.raises(ValueError, match="one dtype"):
        B.tensor_list([torch.zeros(4), torch.zeros(4, dtype=torch.float16)])
    with pytest.raises(ValueError, match="one dtype"):
        B.tensor_list([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError, match="expected"):
        B.tensor_list(g, [torch.zeros(5)], exp_avg=m, exp_avg_sq=m)
    with pytest.raises(ValueError, match="contiguous"):
        B.tensor_list([torch.zeros(4, 4).t()[:, :2]])
    with pytest.raises(ValueError, match="avg_scale"):
        B.tensor_list(g, m, exp_avg=[torch.zeros(4, dtype=torch.uint8)],
                      exp_avg_sq=[torch.zeros(4, dtype=torch.uint8)])
    for kw, msg in ((dict(state_bits=16), "state_bits"), (dict(rounding="up"), "rounding"),
                    (dict(check_finite=False, max_grad_norm=1.0), "check_finite"),
                    (dict(check_finite=False, scale_interval=2), "check_finite"), ({}, "device tensors")):
        with pytest.raises(ValueError, match=msg):
            TensorAdam(m, g, **kw)
    with pytest.raises(ValueError, match="empty"):
        TensorAdam([], [])


@pytest.mark.timeout(600)
def test_under_asan_ubsan():
    if os.environ.get("LD_PRELOAD"):
        pytest.skip("LD_PRELOAD is already set by the environment; the sanitizer runtime must come first")
    from zero_partitioned_mixed_buffer_amd import hostcheck_build
    lib = hostcheck_build.build()
    env = dict(os.environ, LD_PRELOAD=hostcheck_build.runtime(), ZERO_DP_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    env.pop("PYTEST_ADDOPTS", None)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-k",
                        "plan or refusals", os.path.abspath(__file__)],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=540)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0 and " passed" in r.stdout and "runtime error" not in out, out
