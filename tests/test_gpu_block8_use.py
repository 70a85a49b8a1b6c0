"""The 8-bit layer operators as a program uses them: a layer's training step
with TensorAdam, weights out of the gather, captured graphs, several streams,
matrices past 4 GiB, and the binding's refusals."""
import numpy as np
import pytest

from oracle import block8_oracle as bo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
B = pytest.importorskip("zero_partitioned_mixed_buffer_amd.binding")

F32, F64 = np.float32, np.float64
BF = torch.bfloat16
U, HALF = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16


def host(t):
    return t.detach().cpu().double().numpy()


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def held(codes, scales):
    """The float64 values of a matrix in the 8-bit form."""
    return bo.decode(raw(codes), raw(scales))


def workspace(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


class Layer:
    """z = rms_norm(x + r) W^T and its gradients, on buffers made once."""

    def __init__(self, tokens, width, out, dw_type=torch.float32):
        self.shape = (tokens, width, out)

        def new(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        self.h, self.rstd, self.z = new(tokens, width), new(tokens, dtype=torch.float32), new(tokens, out)
        self.y, self.w = B.block8_buffers(tokens, width), B.block8_buffers(out, width, "tiles")
        self.wt, self.yt = B.block8_buffers(width, out, "tiles"), B.block8_buffers(width, tokens)
        self.dz8, self.dzt = B.block8_buffers(tokens, out), B.block8_buffers(out, tokens)
        self.dy, self.dx = new(tokens, width), new(tokens, width)
        self.dw, self.dnorm = new(out, width, dtype=dw_type), new(width, dtype=torch.float32)
        sizes = [B.block8_workspace_bytes(tokens, out, width), B.block8_workspace_bytes(tokens, width, out),
                 B.block8_workspace_bytes(out, width, tokens), B.rms_norm8_workspace_bytes(tokens, width)]
        self.ws = workspace(max(sizes))

    def forward(self, x, r, norm_w, weight):
        B.block8_encode(weight, *self.w, *self.wt, blocks="tiles")
        B.rms_norm8(x, norm_w, *self.y, self.rstd, residual=r, h=self.h)
        B.block8_product(*self.y, *self.w, self.z, workspace=self.ws)
        return self.z

    def backward(self, dz, dh, norm_w, accumulate=False):
        B.block8_encode(dz, *self.dz8, *self.dzt)
        B.block8_product(*self.dz8, *self.wt, self.dy, workspace=self.ws)
        B.block8_encode(self.h, None, None, *self.yt, row_mul=self.rstd, col_mul=norm_w)
        B.block8_product(*self.dzt, *self.yt, self.dw, add=self.dw if accumulate else None, workspace=self.ws)
        B.rms_norm8_backward(self.dy, self.h, norm_w, self.rstd, self.dx, self.dnorm, self.ws, dh=dh)


def layer_inputs(tokens, width, out, seed=0):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g)

    x, r = randn(tokens, width).to(BF).cuda(), (2 * randn(tokens, width)).to(BF).cuda()
    dz, dh = (1e-3 * randn(tokens, out)).to(BF).cuda(), (1e-3 * randn(tokens, width)).to(BF).cuda()
    norm_w, weight = (1 + 0.1 * randn(width)).cuda(), (0.02 * randn(out, width)).cuda()
    return x, r, dz, dh, norm_w, weight


def near(got, want, mag, half=HALF, rel=2.0 ** -10):
    """A product's bound: `rel` of its magnitudes' sum, and half a step of the output."""
    err, tol = np.abs(host(got) - want), half * np.abs(want) + rel * mag + 1e-30
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("tokens,width,out", [(1, 768, 2304), (77, 200, 330), (700, 1600, 512)])
def test_a_layers_step(tokens, width, out):
    """Every stage against float64 on what the stage before it left in memory,
    then TensorAdam on the gradients, against the weights that a float64 AdamW gives."""
    from zero_partitioned_mixed_buffer_amd import TensorAdam
    x, r, dz, dh, norm_w, weight = layer_inputs(tokens, width, out)
    layer = Layer(tokens, width, out)
    z = layer.forward(x, r, norm_w, weight)
    y, w = held(*layer.y), held(*layer.w)
    assert np.array_equal(held(*layer.wt), w.T)
    # the norm's output: half a step of e4m3, or of its smallest normal value under the block's scale (at most
    # 2^-17 of the block's largest magnitude, which the row's root-mean-square bounds by sqrt(width) times the weight)
    want = host(layer.h) * bo.rstd(host(layer.h), 1e-6)[:, None] * host(norm_w)
    assert (np.abs(y - want) <= 1.001 * 2.0 ** -4 * np.abs(want) + 2.0 ** -17 * np.sqrt(width) * 2).all()
    near(z, y @ w.T, np.abs(y) @ np.abs(w).T)

    layer.dw.fill_(1.0)
    layer.backward(dz, dh, norm_w, accumulate=True)
    dz8, dzt, yt = held(*layer.dz8), held(*layer.dzt), held(*layer.yt)
    assert (np.abs(dz8 - host(dz)) <= 2.0 ** -4 * np.abs(host(dz)) + 2.0 ** -17 * np.abs(host(dz)).max()).all()
    assert (np.abs(dzt.T - host(dz)) <= 2.0 ** -4 * np.abs(host(dz)) + 2.0 ** -17 * np.abs(host(dz)).max()).all()
    assert (np.abs(yt.T - want) <= 1.001 * 2.0 ** -4 * np.abs(want) + 2.0 ** -17 * np.sqrt(width) * 2).all()
    near(layer.dy, dz8 @ w, np.abs(dz8) @ np.abs(w))
    # fp32: exact products, each of `tokens` additions off by at most a step
    near(layer.dw, 1.0 + dzt @ yt.T, 1.0 + np.abs(dzt) @ np.abs(yt).T, half=U, rel=(tokens + 2) * 2.0 ** -23)
    dx, dnorm = bo.norm_backward(host(layer.dy), host(layer.h), host(norm_w), host(layer.rstd), host(dh))
    mag = np.abs(host(layer.dy) * host(norm_w)) * host(layer.rstd)[:, None]
    assert (np.abs(host(layer.dx) - dx) <= HALF * np.abs(dx) + 64 * U * (mag + mag.mean(1, keepdims=True) * 10)).all()
    xh = np.abs(host(layer.h)) * host(layer.rstd)[:, None]
    assert (np.abs(host(layer.dnorm) - dnorm) <= (tokens + 4) * U * (np.abs(host(layer.dy)) * xh).sum(0) + U).all()

    before = [host(weight), host(norm_w)]
    opt = TensorAdam([weight, norm_w], [layer.dw, layer.dnorm], lr=1e-2, weight_decay=0.1)
    opt.step()
    for p, old, grad in zip((weight, norm_w), before, (layer.dw, layer.dnorm)):
        gr = host(grad)
        want = old * (1 - 1e-3) - 1e-2 * gr / (np.abs(gr) + 1e-8)  # the first step: m/(1-b1) = g, v/(1-b2) = g^2
        assert (np.abs(host(p) - want) <= 1e-5 * np.abs(want) + 1e-7).all()
    layer.forward(x, r, norm_w, weight)  # and the next step's weights
    assert np.array_equal(raw(layer.w[0]), bo.encode(host(weight).astype(F32), True)[0])


def test_weights_out_of_the_gather():
    """A layer's fp16 weights, gathered from the owners' windows, encoded and used."""
    out, width, part = 130, 200, 16384
    flat = (0.02 * torch.randn(2 * part, generator=torch.Generator().manual_seed(1))).half().cuda()
    lo = 640
    layer = torch.zeros(out * width, dtype=torch.float16, device="cuda")
    B.gather_params([flat[:part], flat[part:]], part, lo, lo + out * width, layer)
    w = B.block8_buffers(out, width, "tiles")
    B.block8_encode(layer.view(out, width), *w, blocks="tiles")
    want = bo.encode(host(flat[lo:lo + out * width]).reshape(out, width), True)
    assert np.array_equal(raw(w[0]), want[0]) and np.array_equal(raw(w[1]), want[1])


def test_weight_gradient_agrees_with_differences():
    """sum(z dz) is linear in the held weights: its differences are exact up to
    the product's own bound."""
    tokens, width, out = 40, 130, 70
    x, r, dz, dh, norm_w, weight = layer_inputs(tokens, width, out, 5)
    layer = Layer(tokens, width, out)
    layer.forward(x, r, norm_w, weight)
    layer.backward(dz, dh, norm_w)
    y, dz8 = held(*layer.y), host(dz)
    for o, c in ((0, 0), (69, 129), (33, 7)):
        e = np.zeros((out, width))
        e[o, c] = 1.0
        diff = ((y @ e.T) * dz8).sum()  # (loss(W + e) - loss(W)) / 1
        # both factors of each product in 8 bits: half a step each, twice over (y by rows and by columns)
        mag = (np.abs(y[:, c]) * np.abs(dz8[:, o])).sum()
        assert abs(host(layer.dw)[o, c] - diff) <= 3 * 2.0 ** -4 * mag + 1e-9


@pytest.mark.parametrize("tokens,width,out", [(3, 300, 520), (9000, 256, 140)])
def test_captured_layer(tokens, width, out):
    """Forward and backward in one graph (a product whose k is split among them),
    replayed on other inputs with eager work between, gives the eager results."""
    args = layer_inputs(tokens, width, out)
    still = [a.clone() for a in args]
    layer, eager = Layer(tokens, width, out), Layer(tokens, width, out)
    assert (B.block8_workspace_bytes(out, width, tokens) > 0) == (tokens > 1000)

    def run(la, x, r, dz, dh, norm_w, weight):
        la.forward(x, r, norm_w, weight)
        la.backward(dz, dh, norm_w)

    run(layer, *still)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(layer, *still)
    for seed in range(1, 5):
        new = layer_inputs(tokens, width, out, seed)
        for s, n in zip(still, new):
            s.copy_(n)
        layer.ws.fill_(0xFF)
        graph.replay()
        run(eager, *new)
        torch.cuda.synchronize()
        for name in ("z", "dx", "dw", "dnorm", "h", "rstd"):
            assert torch.equal(getattr(layer, name), getattr(eager, name)), (seed, name)
        for name in ("y", "w", "wt", "yt", "dz8", "dzt"):
            for a, b in zip(getattr(layer, name), getattr(eager, name)):
                assert np.array_equal(raw(a), raw(b)), (seed, name)


def test_layers_on_two_streams():
    """Two layers at once, each on a stream and a workspace of its own, with
    tensors made on the default stream."""
    sizes = (300, 768, 520)
    a, b = layer_inputs(*sizes, 1), layer_inputs(*sizes, 2)
    want = []
    for args in (a, b):
        la = Layer(*sizes)
        la.forward(args[0], args[1], args[4], args[5])
        la.backward(args[2], args[3], args[4])
        want.append(la)
    la, lb = Layer(*sizes), Layer(*sizes)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for layer, args, st in ((la, a, streams[0]), (lb, b, streams[1])):
            with torch.cuda.stream(st):
                layer.forward(args[0], args[1], args[4], args[5])
                layer.backward(args[2], args[3], args[4])
    torch.cuda.synchronize()
    for got, ref in ((la, want[0]), (lb, want[1])):
        for name in ("z", "dx", "dw", "dnorm"):
            assert torch.equal(getattr(got, name), getattr(ref, name)), name


def test_stream_argument():
    x = torch.randn(300, 400, device="cuda").to(BF)
    c, s = B.block8_buffers(300, 400)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for stream in (st, st.cuda_stream):
        c.view(torch.uint8).zero_()
        torch.cuda.synchronize()
        B.block8_encode(x, c, s, stream=stream)
        st.synchronize()
        assert np.array_equal(raw(c), bo.encode(host(x))[0])


def test_same_call_same_bits():
    """Split sums and gradients have a fixed order."""
    m, n, k = 768, 300, 16000
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = B.block8_buffers(m, k), B.block8_buffers(n, k)
    B.block8_encode(torch.randn(m, k, generator=g, device="cuda"), *a)
    B.block8_encode(torch.randn(n, k, generator=g, device="cuda"), *b)
    assert B.block8_workspace_bytes(m, n, k) > 0
    outs = []
    for _ in range(3):
        out = torch.empty(m, n, device="cuda")
        B.block8_product(*a, *b, out, workspace=workspace(B.block8_workspace_bytes(m, n, k)))
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ------------------------------------------------------- past 4 GiB and 2^32
def test_long_encode_and_norm():
    """5e9 elements: the first and last rows, and the transposed matrix' ends."""
    rows, cols = 76000, 65536 + 16
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    ends = [0, 1, rows - 129, rows - 2, rows - 1]
    x.fill_(1.5)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in ends:
        x[i] = torch.randn(cols, generator=g, device="cuda").to(BF)
    c, s = B.block8_buffers(rows, cols)
    ct, st = B.block8_buffers(cols, rows)
    B.block8_encode(x, c, s, ct, st)
    codes, e = bo.encode(host(x[ends]))
    assert np.array_equal(raw(c[ends]), codes) and np.array_equal(raw(s.view(torch.uint8)[ends]), e)
    for lo, hi in ((0, 128), (cols - 16, cols)):
        sub = host(x[-(rows % 128 or 128):, lo:hi]).T
        codes, e = bo.encode(sub)
        assert np.array_equal(raw(ct[lo:hi, -sub.shape[1]:]), codes)
        assert np.array_equal(raw(st.view(torch.uint8)[lo:hi, -1:]), e)
    del ct, st
    torch.cuda.empty_cache()
    w = torch.randn(cols, generator=g, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    B.rms_norm8(x, w, c, s, rstd, residual=x, h=x)  # x + x in place
    h = host(x[ends])
    assert np.allclose(host(rstd)[ends], bo.rstd(h, 1e-6), rtol=1.1 * U)
    codes, e = bo.encode(bo.normed(h, host(rstd)[ends], host(w)))
    assert np.array_equal(raw(c[ends]), codes) and np.array_equal(raw(s.view(torch.uint8)[ends]), e)


@pytest.mark.parametrize("kind", [torch.float32, BF])
def test_long_product(kind):
    """5.2e9 codes of a, and an out whose rows lie far apart: whole numbers, exact."""
    m, n, k = 80000, 70, 65536
    g = torch.Generator(device="cuda").manual_seed(2)
    a, sa = B.block8_buffers(m, k)
    b, sb = B.block8_buffers(n, k)
    a.view(torch.uint8).fill_(0x38)  # ones
    sa.view(torch.uint8).fill_(127)
    sb.view(torch.uint8).fill_(127)
    ends = [0, 5, m - 300, m - 1]
    for i in ends:
        a[i] = torch.randint(-2, 3, (k,), generator=g, device="cuda").float().to(a.dtype)
    b.copy_(torch.randint(-2, 3, (n, k), generator=g, device="cuda").float().to(b.dtype))
    out = torch.full((m, 30000), 7.0, dtype=kind, device="cuda")
    B.block8_product(a, sa, b, sb, out[:, 29000:29070], workspace=workspace(B.block8_workspace_bytes(m, n, k)))
    want = (a[ends].double() @ b.double().t()).to(kind)
    assert torch.equal(out[ends, 29000:29070], want)
    rest = b.double().sum(1).to(kind)
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[ends] = False
    assert bool((out[keep, 29000:29070] == rest).all())
    assert bool((out[:, :29000] == 7).all()) and bool((out[:, 29070:] == 7).all())


@pytest.mark.parametrize("m,n", [(20, 30), (300, 200), (200, 2100)])
def test_product_of_rows_far_apart(m, n):
    """The longest strides: rows of codes 2^23 bytes apart, scales 2^20."""
    k = 200
    g = torch.Generator(device="cuda").manual_seed(4)

    def far(rows):
        c = torch.full((rows, 1 << 23), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :k]
        s = torch.full((rows, 1 << 20), 0xFF, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)[:, :2]
        c.copy_(torch.randint(-2, 3, (rows, k), generator=g, device="cuda").float().to(c.dtype))
        s.view(torch.uint8).fill_(127)
        return c, s

    (a, sa), (b, sb) = far(m), far(n)
    want = a.double() @ b.double().t()
    for kind in (torch.float32, BF):
        out = torch.empty(m, n, dtype=kind, device="cuda")
        B.block8_product(a, sa, b, sb, out, workspace=workspace(B.block8_workspace_bytes(m, n, k)))
        assert torch.equal(out, want.to(kind))


@pytest.mark.parametrize("cols", [100003, 1 << 20])
def test_rows_longer_than_registers(cols):
    rows = 3
    x, r = torch.randn(rows, cols, device="cuda"), torch.randn(rows, cols, device="cuda")
    w, dy = torch.rand(cols, device="cuda") + 0.5, 1e-3 * torch.randn(rows, cols, device="cuda")
    c, s = B.block8_buffers(rows, cols)
    rstd, h = torch.empty(rows, device="cuda"), torch.empty_like(x)
    B.rms_norm8(x, w, c, s, rstd, residual=r, h=h)
    assert torch.equal(h, x + r)
    assert np.allclose(host(rstd), bo.rstd(host(h), 1e-6), rtol=1.1 * U)
    codes, e = bo.encode(bo.normed(host(h), host(rstd), host(w)))
    assert np.array_equal(raw(c), codes) and np.array_equal(raw(s), e)
    dx, dw = torch.empty_like(x), torch.empty(cols, device="cuda")
    B.rms_norm8_backward(dy, h, w, rstd, dx, dw, workspace(B.rms_norm8_workspace_bytes(rows, cols)))
    want, want_w = bo.norm_backward(host(dy), host(h), host(w), host(rstd))
    xh, gg = np.abs(host(h) * host(rstd)[:, None]), np.abs(host(dy) * host(w))
    depth = 8 * -(-cols // 8192) + 22  # a lane's additions, six across its wave, 16 waves
    tol = host(rstd)[:, None] * U * (3 * gg + xh * (gg * xh).mean(1, keepdims=True) * (depth + 9)) + 2 * U * np.abs(want)
    assert (np.abs(host(dx) - want) <= tol).all()
    assert (np.abs(host(dw) - want_w) <= (rows + 4) * U * (np.abs(host(dy)) * xh).sum(0) + U * np.abs(want_w)).all()


# --------------------------------------------------------------- refusals
def test_binding_refusals():
    d = "cuda"
    x, w, rstd = torch.randn(20, 300, device=d).to(BF), torch.ones(300, device=d), torch.empty(20, device=d)
    c, s = B.block8_buffers(20, 300)
    t, ts = B.block8_buffers(20, 300, "tiles")

    def refused(f, *a, **k):
        with pytest.raises((ValueError, B.ZeroError)):
            f(*a, **k)

    enc, norm, back, prod = B.block8_encode, B.rms_norm8, B.rms_norm8_backward, B.block8_product
    refused(enc, x)
    refused(enc, x, c)
    refused(enc, x, c, s, blocks="columns")
    refused(enc, x.cpu(), c, s)
    refused(enc, x, c.cpu(), s)
    refused(enc, x.double(), c, s)
    refused(enc, x[0], c, s)
    refused(enc, x.t(), c, s)
    refused(enc, x[:, ::2], *B.block8_buffers(20, 150))
    refused(enc, x[:1].expand(20, 300), c, s)
    refused(enc, x, c, ts)
    refused(enc, x, t, ts, blocks="rows")
    refused(enc, x, c, s[:, :2])
    refused(enc, x, c[:, 1:], s)
    refused(enc, x[:, 1:], c[:, 1:], s)  # codes off their 16 bytes
    refused(enc, x, torch.empty(20, 300, dtype=torch.float8_e4m3fn, device=d), s)  # rows 300 bytes apart
    refused(enc, x, c, s, row_mul=w)
    refused(enc, x, c, s, row_mul=rstd.half())
    refused(enc, x, c, s, col_mul=rstd)
    refused(enc, x, c, s, col_mul=torch.ones(600, device=d)[::2])
    refused(norm, x, w[:299], c, s, rstd)
    refused(norm, x, w, t, ts, rstd)
    refused(norm, x, w, c, s, rstd[:19])
    refused(norm, x, w, c, s, rstd, residual=x.clone())
    refused(norm, x, w, c, s, rstd, h=x.clone())
    refused(norm, x, w, c, s, rstd, residual=x.float(), h=x.clone())
    refused(norm, x, w, c, s, rstd, eps=0.0)
    refused(norm, x, w.double(), c, s, rstd)
    refused(norm, x, w, c, s, rstd, residual=x.clone(), h=torch.empty(21, 300, dtype=BF, device=d)[1:].t().t()[:19])
    ws = workspace(B.rms_norm8_workspace_bytes(20, 300))
    dw, dx = torch.empty(300, device=d), torch.empty_like(x)
    refused(back, x, x.clone(), w, rstd, dx, dw)  # no workspace
    refused(back, x, x.clone(), w, rstd, dx, dw, ws[:-16])
    refused(back, x, x.clone(), w, rstd, dx, dw.half(), ws)
    refused(back, x, x.float(), w, rstd, dx, dw, ws)
    hh = x.clone()
    refused(back, x, hh, w, rstd, hh, dw, ws)  # dx over h
    out = torch.empty(20, 20, dtype=BF, device=d)
    refused(prod, c, s, c, s, out[:19])
    refused(prod, c, s, c[:, :200], s[:, :2], out)
    refused(prod, c, s, c, s, out, add=out.float())
    refused(prod, c, s, c, s, out.to(torch.int16))
    refused(prod, c, s, c, s, out.t())
    k = 32768
    a, sa = B.block8_buffers(100, k)
    big = torch.empty(100, 100, dtype=BF, device=d)
    refused(prod, a, sa, a, sa, big)  # no workspace
    refused(prod, a, sa, a, sa, big, workspace=torch.empty(8, device=d))
    refused(prod, a, sa, a, sa, big, workspace=workspace(B.block8_workspace_bytes(100, 100, k)).cpu())
    refused(B.block8_buffers, -1, 5)
    refused(B.block8_buffers, 5, 5, "columns")


def test_autograd_sees_what_is_written():
    """A backward pass through a graph that saved a tensor which a call then wrote
    raises, as after torch's own in-place operations."""
    def saved(*shape):
        w = torch.ones(shape, device="cuda", requires_grad=True)
        a = w * 2
        return a.detach(), (a * w).sum()

    w, rstd = torch.ones(128, device="cuda"), torch.ones(64, device="cuda")
    x, (c, s) = torch.randn(64, 128, device="cuda"), B.block8_buffers(64, 128)
    ws = workspace(B.rms_norm8_workspace_bytes(64, 128))
    calls = []
    a, loss = saved(64, 128)
    B.rms_norm8(x, w, c, s, rstd, residual=a, h=a)
    calls.append(loss)
    a, loss = saved(64, 128)
    B.rms_norm8_backward(x, x.clone(), w, rstd, a, torch.empty(128, device="cuda"), ws)
    calls.append(loss)
    a, loss = saved(128)
    B.rms_norm8_backward(x, x.clone(), w, rstd, torch.empty_like(x), a, ws)
    calls.append(loss)
    a, loss = saved(64, 64)
    B.block8_product(c, s, c, s, a)
    calls.append(loss)
    for loss in calls:
        with pytest.raises(RuntimeError):
            loss.backward()


def test_results_are_bytes_too():
    """uint8 tensors serve as codes and scales."""
    x = torch.randn(33, 200, device="cuda")
    c, s = B.block8_buffers(33, 200)
    B.block8_encode(x, c.view(torch.uint8), s.view(torch.uint8))
    assert np.array_equal(raw(c), bo.encode(host(x))[0]) and np.array_equal(raw(s), bo.encode(host(x))[1])
