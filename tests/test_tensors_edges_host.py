"""Host-side checks (no GPU) of the tensor lists' 8-bit form at the ends of
its range: the oracle that the GPU tests compare with."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import tensor_oracle as to

F32 = np.float32


def test_no_finite_value_reads_back_as_inf():
    """Over the largest scale, 2^120, codes end at 240."""
    x = np.full(64, 1e30, F32)
    x[:3] = np.finfo(F32).max, -np.finfo(F32).max, 3.2e38
    for words in (None, np.full(64, 0xFFFFFFFF)):
        codes, scales = to.mx8_encode(x, words=words)
        y = to.mx8_decode(codes, scales)
        assert scales[0] == 247 and y[:3].tolist() == [240 * 2.0 ** 120, -240 * 2.0 ** 120, 240 * 2.0 ** 120]
        assert np.isfinite(y).all()
        for root in (False, True):  # the root of the largest float is far from the end
            assert np.isfinite(to.mx8_decode(*to.mx8_encode(np.abs(x), root, words))).all()


# ------------------------------------------------- the random part of a root
ALL16 = np.arange(1 << 16, dtype=np.uint64)


def _codes_over_all_words(root, top):
    """Codes of the root `root` in a block whose largest is `top`, under each
    of the 2^16 random parts, and its value in the code's steps."""
    many = np.full((1 << 16, 32), F32(root), F32)
    many[:, 31] = F32(top)
    words = np.zeros((1 << 16, 32), np.uint64)
    words[:, 0] = ALL16 | np.uint64(0xABCD0000)  # a root does not look at the upper half
    codes, e = to.mx8_encode(many.reshape(-1), True, words.reshape(-1), taken=True)
    y = Fraction(float(F32(root))) / Fraction(2) ** (int(e[0]) - 127)
    step = Fraction(2) ** (max(int(np.floor(np.log2(float(y)))), -6) - 3)
    vals = to.code_values()[codes.reshape(-1, 32)[:, 0]]
    return vals / float(step), y / step


@pytest.mark.parametrize("top,root", [(448.0, 3.3), (448.0, 0.01), (300.0, 17.77), (2.0 ** -100, 1.7e-31),
                                      (448.0, 8.0), (448.0, 8.0 + 2.0 ** -18)])
def test_stochastic_roots_round_up_in_steps_of_2_to_the_minus_16(top, root):
    got, y = _codes_over_all_words(root, top)
    low = y.__floor__()
    assert np.isin(got, (low, low + 1)).all()
    # floor(y + R/2^16) is up iff R >= 2^16 (1 - frac)
    assert int((got > low).sum()) == ((1 << 16) * (y - low)).__floor__()


@pytest.mark.parametrize("beta2", [0.99, 0.999, 0.9999])
def test_stochastic_roots_decay_at_the_stated_rate(beta2):
    """Over all random parts the mean of a decayed root falls short of its
    value by less than 2^-16 of a code's step (and half an fp32 rounding of
    the root, 2^-24 of at most 16 steps), so the decay is too fast by less
    than 2^-18 / (1 - beta2) of itself."""
    for k in range(8, 16):
        r = F32(k)
        new = np.sqrt(F32(beta2 * float(r) ** 2))
        got, _ = _codes_over_all_words(new, 240.0)
        got = got * (0.5 if new < 8 else 1.0)  # steps of 8..16, whose size is 1
        want = float(r) * np.sqrt(beta2)
        short = want - got.mean()
        assert -2.0 ** -20 <= short < 2.0 ** -16 + 2.0 ** -20
        assert short / (float(r) - want) < 1.07 * 2.0 ** -18 / (1 - beta2)
