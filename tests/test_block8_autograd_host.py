"""The 8-bit layer operators and autograd (no GPU): it records none of these
calls, so a tensor that requires a gradient is refused while it records.  The
library is replaced by a stub that takes every call."""
import pytest

torch = pytest.importorskip("torch")
B = pytest.importorskip("zero_partitioned_mixed_buffer_amd.binding")


class Stub:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def stub(monkeypatch):
    s = Stub()
    monkeypatch.setattr(B, "lib", lambda: s)
    monkeypatch.setattr(B, "_current_device", lambda: -1)  # get_device() of tensors in host memory
    return s


def operands():
    """For each call, its tensors by name (a new set each time)."""
    m, n, k = 8, 16, 32

    def mat(r, c):
        return torch.zeros(r, c)

    c, s = B.block8_buffers(m, k, device="cpu")
    ct, st = B.block8_buffers(k, m, device="cpu")
    bc, bs = B.block8_buffers(n, k, device="cpu")
    return {
        "block8_encode": dict(x=mat(m, k), codes=c, scales=s, codes_t=ct, scales_t=st, row_mul=torch.ones(m),
                              col_mul=torch.ones(k)),
        "rms_norm8": dict(x=mat(m, k), weight=torch.ones(k), codes=c, scales=s, rstd=torch.ones(m),
                          residual=mat(m, k), h=mat(m, k)),
        "rms_norm8_backward": dict(dy=mat(m, k), h=mat(m, k), weight=torch.ones(k), rstd=torch.ones(m), dx=mat(m, k),
                                   dweight=torch.ones(k), dh=mat(m, k)),
        "block8_product": dict(a=c, a_scales=s, b=bc, b_scales=bs, out=mat(m, n), add=mat(m, n)),
    }


CALLS = [(f, name) for f, names in operands().items() for name, t in names.items() if t.dtype == torch.float32]


@pytest.mark.parametrize("f,name", CALLS)
def test_refused_while_autograd_records(stub, f, name):
    args = operands()[f]
    args[name].requires_grad_()
    version = {k: t._version for k, t in args.items()}
    with pytest.raises(ValueError, match="requires a gradient"):
        getattr(B, f)(**args, stream=0)
    assert "zero_" + f not in stub.calls and version == {k: t._version for k, t in args.items()}


@pytest.mark.parametrize("f", ["block8_encode", "rms_norm8", "rms_norm8_backward", "block8_product"])
def test_taken_where_nothing_is_recorded(stub, f):
    for name in [n for g, n in CALLS if g == f]:
        args = operands()[f]
        args[name].requires_grad_()
        with torch.no_grad():
            getattr(B, f)(**args, stream=0)
        args[name] = args[name].detach()
        getattr(B, f)(**args, stream=0)
    assert stub.calls.count("zero_" + f) == 2 * len([n for g, n in CALLS if g == f])


def test_a_parameters_gradient_through_a_function(stub):
    """The way to gradients: a function whose passes are these calls."""
    class Encode(torch.autograd.Function):
        @staticmethod
        def forward(ctx, w):
            c, s = B.block8_buffers(*w.shape, device="cpu")
            B.block8_encode(w, c, s, stream=0)
            return w.new_ones(())

        @staticmethod
        def backward(ctx, d):
            return torch.full((8, 32), 3.0)

    w = torch.nn.Parameter(torch.zeros(8, 32))
    Encode.apply(w).backward()
    assert stub.calls == ["zero_block8_encode"] and bool((w.grad == 3).all())
