"""The tensor-list operators on the GPU at the ends of their ranges and in
calls that the parity tests do not make: against the oracle where it applies,
with the bounds derived at the head of test_gpu_tensors.py.
"""
import pytest

from test_gpu_tensors import Lists

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ top of the range
@pytest.mark.parametrize("beta2", [0.999, 0.5])
@pytest.mark.parametrize("kind,value", [("f32", 1e38), ("f32", 3e38), ("bf16", 1e38), ("bf16", 3e38)])
def test_gradients_near_the_top_of_the_range(kind, value, beta2):
    """Denominators above 2^126, whose reciprocals are denormal: the weight
    moves by about lr, as the formula says."""
    x = Lists([40, 4097, 5000], kind, "bf16", True, seed=31, beta2=beta2)
    for t in range(16):
        before = float(x.p[1][70])
        assert x.step(poison=(1, 70, value if t != 9 else -value))["overflow"] == 0
        x.check(t)
        if t == 0:  # m'/(1-b1) = r/sqrt(1-b2) = g; the decay of a weight below 0.1 is below 1e-6
            assert abs(before - float(x.p[1][70]) - 1e-3) < 2e-6
    assert all(bool(p.isfinite().all()) for p in x.p)


@pytest.mark.parametrize("eps", [1e38, 1e39])
def test_eps_past_the_range(eps):
    x = Lists([40, 4097], "f32", None, True, seed=32, eps=eps)
    for t in range(3):
        x.step(poison=(1, 70, 3e38))
        x.check(t)
