"""Host-side checks (no GPU) of the tensor lists' 8-bit form at the ends of
its range: the oracle that the GPU tests compare with."""
import numpy as np

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
