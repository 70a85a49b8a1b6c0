"""The 8-bit product's sums and kernels on the GPU: what its 16-bit outputs are
off by, at the ends of the codes' range and over long k."""
import numpy as np
import pytest

from oracle import block8_oracle as bo
from test_gpu_block8 import DT, HALF, LEAST, Guarded, _ints, _ws, host, raw

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
B = pytest.importorskip("zero_partitioned_mixed_buffer_amd.binding")

F32, F64 = np.float32, np.float64


# ------------------------------------------------------- sums of 16-bit outputs
def sum_bound(k):
    """Of the sum of the products' magnitudes, each factor counted as at least
    2^-6 of its scale: eight neighbouring k share a unit, 2^-13 of the largest
    product's power of two (a factor below the smallest normal code has that
    code's exponent), and seven of them are cut at it; then at most k / 16
    additions to the accumulator and one before each, 256 parts or 8 waves'
    sums, each off by at most a step of fp32."""
    return 7 * 2.0 ** -13 + (k / 16 + 258) * 2.0 ** -23


def on_device(codes, e, tiles=False):
    """Host codes and scale bytes as device tensors, their values and the values
    of which none is below 2^-6 of its scale."""
    c, s = B.block8_buffers(*codes.shape, blocks="tiles" if tiles else "rows")
    c.view(torch.uint8).copy_(torch.from_numpy(codes))
    s.view(torch.uint8).copy_(torch.from_numpy(e))
    v = bo.decode(codes, e)
    scale = bo.decode(np.full_like(codes, 0x38), e)  # code 1.0
    return c, s, torch.from_numpy(v).cuda(), torch.from_numpy(np.maximum(np.abs(v), scale * 2.0 ** -6)).cuda()


def code_of(x):
    return torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def check_sums(a, b, k, kind):
    """A product's values against float64, with the bound's share that they take."""
    (ca, sa, av, am), (cb, sb, bv, bm) = a, b
    m, n = ca.shape[0], cb.shape[0]
    want, mag = av @ bv.t(), am @ bm.t()
    out = torch.empty(m, n, dtype=DT[kind], device="cuda")
    B.block8_product(ca, sa, cb, sb, out, workspace=_ws(m, n, k))
    err = (out.double() - want).abs()
    tol = HALF[kind] * want.abs() + LEAST[kind] + sum_bound(k) * mag
    assert bool((err <= tol).all()), float((err / tol).max())
    exact = torch.empty(m, n, device="cuda")  # the way to sums in fp32
    B.block8_product(ca, sa, cb, sb, exact, workspace=_ws(m, n, k))
    assert bool(((exact.double() - want).abs() <= (k + 2) * 2.0 ** -23 * (av.abs() @ bv.abs().t())).all())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(16, 40, 1000), (2300, 800, 1000), (4100, 4100, 200)])
def test_sums_of_codes_below_the_normal_ones(m, n, k, kind):
    """Groups whose largest product is 2^-9 * 448, or whose only large factor meets
    a zero, with seven small ones of one sign beside it: the share that is cut
    there is far more than 2^-10 of the true magnitudes."""
    g = np.random.default_rng(1)
    x, y = np.full((m, k), 2.0 ** -6), np.full((n, k), 2.0 ** -6)
    at = np.arange(0, k, 8)
    x[:, at] = g.choice([2.0 ** -9, -(2.0 ** -9), 0.0, 3 * 2.0 ** -9], (m, len(at)))
    y[:, at] = g.choice([448.0, 256.0, 1.0], (n, len(at)))
    e = np.full((m, bo.blocks_of(k)), 127, np.uint8)
    f = g.integers(120, 130, (n, bo.blocks_of(k))).astype(np.uint8)
    check_sums(on_device(code_of(x), e), on_device(code_of(y), f), k, kind)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(3, 20, 1 << 20), (300, 200, 1 << 17), (130, 140, (1 << 17) + 77)])
def test_sums_over_long_k(m, n, k, kind):
    """Over 131072 and more k, of one sign (every addition rounds the same large
    sum) and of both."""
    g = np.random.default_rng(2)
    for sign in (1, -1):
        codes = [g.integers(1, 0x40, (r, k)).astype(np.uint8) for r in (m, n)]
        if sign < 0:
            codes = [c | (g.integers(0, 2, c.shape) * 128).astype(np.uint8) for c in codes]
        es = [g.integers(112, 116, (r, bo.blocks_of(k))).astype(np.uint8) for r in (m, n)]
        check_sums(*(on_device(c, e) for c, e in zip(codes, es)), k, kind)
