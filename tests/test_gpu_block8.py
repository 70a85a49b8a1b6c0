"""The 8-bit layer operators on the GPU against the float64 oracle: encode, the
root-mean-square norm and its gradients, the product, and a layer's training
step made of them."""
import numpy as np
import pytest

from oracle import block8_oracle as bo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
B = pytest.importorskip("zero_partitioned_mixed_buffer_amd.binding")

F32, F64 = np.float32, np.float64
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24  # half a step of fp32
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}
GUARD = 0x5A


def host(t):
    return t.detach().cpu().double().numpy()


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


class Guarded:
    """A matrix [rows, cols] inside a larger buffer whose other bytes are checked
    afterwards: `pad` elements beside it, a row above and below."""

    def __init__(self, rows, cols, dtype, pad=16, lead=16):
        self.size = torch.empty(0, dtype=dtype).element_size()
        width = lead + cols + pad
        width += -width % 16
        self.box = torch.full((rows + 2, width * self.size), GUARD, dtype=torch.uint8, device="cuda")
        self.view = self.box.view(dtype)[1:rows + 1, lead:lead + cols]
        self.at = (rows, cols * self.size, lead * self.size)

    def check(self):
        rows, n, lead = self.at
        x = self.box.cpu().numpy().copy()
        x[1:rows + 1, lead:lead + n] = GUARD
        assert (x == GUARD).all(), "bytes beside the output were written"


def guarded_block8(rows, cols, blocks="rows"):
    srows = rows if blocks == "rows" else bo.blocks_of(rows)
    return (Guarded(rows, cols, torch.float8_e4m3fn), Guarded(srows, bo.blocks_of(cols), torch.float8_e8m0fnu))


def device_block8(x, tiles=False, pad=0):
    """The oracle's encoding of a host matrix, as device tensors, and the values."""
    codes, e = bo.encode(x, tiles)
    c, s = B.block8_buffers(*codes.shape, blocks="tiles" if tiles else "rows")
    c.view(torch.uint8).copy_(torch.from_numpy(codes))
    s.view(torch.uint8).copy_(torch.from_numpy(e))
    return c, s, bo.decode(codes, e)


def values(g, rows, cols, kind):
    """Blocks of very different sizes, zeros, and values at codes' borders."""
    x = g.standard_normal((rows, cols)) * np.exp2(g.integers(-12, 12, (rows, 1))) * np.exp2(g.integers(-3, 3, (1, cols)))
    x[g.random((rows, cols)) < 0.1] = 0.0
    if rows > 2:
        x[1] = 0.0
    x.flat[0] = 448.0
    x.flat[-1] = -449.0
    return torch.from_numpy(x.astype(F32)).to(DT[kind]).cuda()


SIZES = [(1, 1), (1, 130), (2, 128), (5, 127), (129, 256), (128, 513), (130, 700), (257, 1030)]


# ------------------------------------------------------------------ encode
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_encode_is_the_oracles(rows, cols, blocks, kind):
    """Bit for bit, each of the outputs alone and both together."""
    g = np.random.default_rng(rows * 7 + cols)
    x = values(g, rows, cols, kind)
    want = bo.encode(host(x), blocks == "tiles")
    want_t = bo.encode(host(x).T, blocks == "tiles")
    for outs in ("plain", "turned", "both"):
        c, s = guarded_block8(rows, cols, blocks)
        ct, st = guarded_block8(cols, rows, blocks)
        plain = (c.view, s.view) if outs != "turned" else (None, None)
        turned = (ct.view, st.view) if outs != "plain" else (None, None)
        B.block8_encode(x, *plain, *turned, blocks=blocks)
        if outs != "turned":
            assert np.array_equal(raw(s.view), want[1]), outs
            assert np.array_equal(raw(c.view), want[0]), outs
        if outs != "plain":
            assert np.array_equal(raw(st.view), want_t[1]), outs
            assert np.array_equal(raw(ct.view), want_t[0]), outs
        for t in (c, s, ct, st):
            t.check()


@pytest.mark.parametrize("blocks", ["rows", "tiles"])
def test_encode_of_strided_rows_and_multipliers(blocks):
    g = np.random.default_rng(5)
    x = values(g, 150, 400, "bf16")[:, 3:333]
    rm = torch.from_numpy(np.exp(g.standard_normal(150)).astype(F32)).cuda()
    for cm in (torch.from_numpy(g.standard_normal(330).astype(F32)).cuda(),
               torch.from_numpy(g.standard_normal(330).astype(F32)).half().cuda(), None):
        for use in (rm, None):
            y = host(x).astype(F32)
            y = y if use is None else y * use.cpu().numpy()[:, None]
            y = y if cm is None else y * cm.float().cpu().numpy()
            (c, s), (ct, st) = B.block8_buffers(150, 330, blocks), B.block8_buffers(330, 150, blocks)
            B.block8_encode(x, c, s, ct, st, blocks=blocks, row_mul=use, col_mul=cm)
            for (gc, gs), want in (((c, s), bo.encode(y, blocks == "tiles")), ((ct, st), bo.encode(y.T, blocks == "tiles"))):
                assert np.array_equal(raw(gs), want[1])
                assert np.array_equal(raw(gc), want[0])


@pytest.mark.parametrize("blocks", ["rows", "tiles"])
def test_encode_at_the_ends_of_the_range(blocks):
    """Infinities and NaN blot out their block alone; the largest and smallest
    floats, subnormals and negative zeros."""
    x = np.zeros((300, 300), F32)
    x[0, 0], x[130, 5], x[299, 299], x[5, 200] = np.inf, -np.inf, np.nan, 3.4e38
    x[140:, 128:256] = 1e-45
    x[200, 140:150] = 2.0 ** -126
    x[260:, :100] = -0.0
    x[280, :50] = 1e-40
    d = torch.from_numpy(x).cuda()
    (c, s), (ct, st) = B.block8_buffers(300, 300, blocks), B.block8_buffers(300, 300, blocks)
    B.block8_encode(d, c, s, ct, st, blocks=blocks)
    for (gc, gs), src in (((c, s), x), ((ct, st), x.T)):
        codes, e = bo.encode(src, blocks == "tiles")
        assert np.array_equal(raw(gs), e)
        assert np.array_equal(raw(gc), codes)
    # the blocks that hold an infinity or a NaN, and no others
    bad = {(0, 0), (130, 0), (299, 2)} if blocks == "rows" else {(0, 0), (1, 0), (2, 2)}
    assert set(zip(*np.nonzero(raw(s) == 255))) == bad


# -------------------------------------------------------------------- norm
ROWS = [(1, 1), (3, 8), (5, 127), (9, 512), (6, 513), (5, 1600), (3, 2049), (4, 4100), (3, 8200), (2, 16385), (3, 20001)]


def _norm_inputs(rows, cols, kind, seed):
    g = np.random.default_rng(seed)
    x = torch.from_numpy(g.standard_normal((rows, cols)).astype(F32)).to(DT[kind]).cuda()
    r = torch.from_numpy((3 * g.standard_normal((rows, cols))).astype(F32)).to(DT[kind]).cuda()
    w = torch.from_numpy((1 + 0.3 * g.standard_normal(cols)).astype(F32)).to(DT[kind]).cuda()
    if rows > 2:
        x[1], r[1] = 0, 0  # a row of padding
    return g, x, r, w


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_norm_is_the_oracles(rows, cols, kind):
    g, x, r, w = _norm_inputs(rows, cols, kind, rows + cols)
    for res in (True, False):
        c, s = guarded_block8(rows, cols)
        h = Guarded(rows, cols, DT[kind])
        rstd = torch.full((rows,), -1.0, device="cuda")
        B.rms_norm8(x, w, c.view, s.view, rstd, residual=r if res else None, h=h.view if res else None, eps=1e-5)
        want_h = (x.float() + r.float()).to(DT[kind]) if res else x
        if res:
            assert torch.equal(h.view, want_h)
        # the sum is in float64, rounded to fp32 once
        want = bo.rstd(host(want_h), 1e-5)
        got = host(rstd)
        assert (np.abs(got - want) <= 1.01 * U * want).all()
        codes, e = bo.encode(bo.normed(host(want_h), got, host(w)))
        assert np.array_equal(raw(s.view), e)
        assert np.array_equal(raw(c.view), codes)
        for t in (c, s, h):
            t.check()


def test_norm_in_place_and_weight_types():
    """h may be x or residual itself; the weight has a type of its own."""
    _, x, r, w = _norm_inputs(7, 700, "bf16", 3)
    for wt in (w, w.float(), w.half()):
        outs = []
        for which in range(3):
            a, b = x.clone(), r.clone()
            h = (torch.empty_like(a), a, b)[which]
            c, s = B.block8_buffers(7, 700)
            rstd = torch.empty(7, device="cuda")
            B.rms_norm8(a, wt, c, s, rstd, residual=b, h=h)
            outs.append((h.clone(), raw(c), raw(s), rstd))
        for o in outs[1:]:
            assert torch.equal(o[0], outs[0][0]) and torch.equal(o[3], outs[0][3])
            assert np.array_equal(o[1], outs[0][1]) and np.array_equal(o[2], outs[0][2])
        codes, e = bo.encode(bo.normed(host(outs[0][0]), host(outs[0][3]), host(wt)))
        assert np.array_equal(outs[0][1], codes) and np.array_equal(outs[0][2], e)


@pytest.mark.parametrize("cols", [300, 3000])
def test_norm_of_large_infinite_and_nan_rows(cols):
    x = np.ones((6, cols), F32)
    x[0] = 1e30          # squares past fp32's range
    x[1] = 1e-30         # squares below it
    x[2, 5] = np.inf
    x[3, 200] = np.nan
    x[4] = 0.0
    d, w = torch.from_numpy(x).cuda(), torch.ones(cols, device="cuda")
    c, s = B.block8_buffers(6, cols)
    rstd = torch.empty(6, device="cuda")
    B.rms_norm8(d, w, c, s, rstd, eps=1e-6)
    got = host(rstd)
    want = bo.rstd(x, 1e-6)
    assert np.allclose(got[[0, 1, 4, 5]], want[[0, 1, 4, 5]], rtol=2 * U)
    assert got[2] == 0 and np.isnan(got[3])
    codes, e = bo.encode(bo.normed(x, got, np.ones(cols)))
    assert np.array_equal(raw(c), codes) and np.array_equal(raw(s), e)
    assert (raw(s)[2] == 255).sum() == 1 and (raw(s)[3] == 255).all()


def _depth(cols):
    """Additions one after the other in a row's sum: a lane's own (its units of 8,
    one for every 512, 2048 or 8192 columns), six across a wave, 16 waves."""
    return 8 * max(4, -(-cols // 8192)) + 6 + 16


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", ROWS + [(700, 260), (2600, 40)])
def test_norm_backward_is_the_oracles(rows, cols, kind):
    g, h, dh, w = _norm_inputs(rows, cols, kind, rows + cols + 1)
    dy = torch.from_numpy((1e-2 * g.standard_normal((rows, cols))).astype(F32)).to(DT[kind]).cuda()
    rstd = torch.from_numpy(bo.rstd(host(h), 1e-2).astype(F32)).cuda()
    ws = torch.empty(B.rms_norm8_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda").fill_(0xFF)
    for extra in (dh, None):
        dx = Guarded(rows, cols, DT[kind])
        dw = torch.full((cols,), 7.0, device="cuda")
        B.rms_norm8_backward(dy, h, w, rstd, dx.view, dw, ws, dh=extra)
        want, want_w = bo.norm_backward(host(dy), host(h), host(w), host(rstd), None if extra is None else host(extra))
        r = host(rstd)[:, None]
        xh, gg = np.abs(host(h) * r), np.abs(host(dy) * host(w))
        mean = (gg * xh).mean(axis=1, keepdims=True)
        # c: products of two rounded factors, `depth` additions, one division
        tol = r * U * (3 * gg + xh * mean * (_depth(cols) + 4 + 5)) + U * np.abs(want) + HALF[kind] * np.abs(want) + LEAST[kind]
        err = np.abs(host(dx.view) - want)
        assert (err <= tol).all(), float((err / tol).max())
        dx.check()
        # products of a rounded factor, and at most `rows` additions
        tol_w = (rows + 4) * U * (np.abs(host(dy)) * xh).sum(axis=0) + U * np.abs(want_w)
        err = np.abs(host(dw) - want_w)
        assert (err <= tol_w).all(), float((err / tol_w).max())
        # in place, and without dweight
        for into in ("dy", "dh"):
            if into == "dh" and extra is None:
                continue
            a, b = dy.clone(), None if extra is None else extra.clone()
            B.rms_norm8_backward(a, h, w, rstd, a if into == "dy" else b, dh=b)
            assert torch.equal(a if into == "dy" else b, dx.view)


def test_norm_backward_agrees_with_differences():
    """d(sum of y dy) / dx and / dw by central differences in float64."""
    g = np.random.default_rng(11)
    h, dy, w = g.standard_normal((4, 50)), g.standard_normal((4, 50)), 1 + 0.2 * g.standard_normal(50)
    f32 = [torch.from_numpy(a.astype(F32)).cuda() for a in (dy, h, w)]
    rstd = torch.from_numpy(bo.rstd(f32[1].cpu().numpy(), 1e-6).astype(F32)).cuda()
    dx, dw = torch.empty(4, 50, device="cuda"), torch.empty(50, device="cuda")
    ws = torch.empty(B.rms_norm8_workspace_bytes(4, 50), dtype=torch.uint8, device="cuda")
    B.rms_norm8_backward(*f32[:2], f32[2], rstd, dx, dw, ws)
    dy, h, w = (host(t) for t in f32)

    def loss(h, w):
        return (h * bo.rstd(h, 1e-6)[:, None] * w * dy).sum()

    d = 1e-5  # differences err by d^2 and 2^-53 / d: both far below 1e-6
    for got, at in ((dx, 0), (dw, 1)):
        got = host(got)
        for k in np.ndindex(got.shape):
            p, m = [h.copy(), w.copy()], [h.copy(), w.copy()]
            p[at][k] += d
            m[at][k] -= d
            diff = (loss(*p) - loss(*m)) / (2 * d)
            assert abs(diff - got[k]) <= 1e-5 * (1 + abs(diff))


def test_norm_of_no_rows():
    w = torch.ones(40, device="cuda")
    none = torch.empty(0, 40, device="cuda")
    c, s = B.block8_buffers(0, 40)
    B.rms_norm8(none, w, c, s, torch.empty(0, device="cuda"))
    dw = torch.full((40,), 3.0, device="cuda")
    B.rms_norm8_backward(none, none, w, torch.empty(0, device="cuda"), none.clone(), dw)
    assert (dw == 0).all()


# ----------------------------------------------------------------- product
MNK = [(1, 1, 1), (1, 16, 128), (1, 200, 1600), (3, 5, 7), (16, 33, 129), (17, 64, 512), (33, 100, 300), (64, 130, 2000),
       (65, 130, 257), (127, 129, 640), (200, 300, 1000), (300, 20, 4096), (130, 140, 8200), (2900, 2900, 200),
       (4000, 2100, 128), (70, 3, 16)]


def _ints(g, rows, cols, tiles):
    """Small whole numbers under scales of 1/2 to 2: every product and sum over
    k is exact in the instructions' arithmetic and in fp32."""
    codes = torch.from_numpy(g.integers(-4, 5, (rows, cols)).astype(F32)).to(torch.float8_e4m3fn)
    srows = bo.blocks_of(rows) if tiles else rows
    e = g.integers(126, 129, (srows, bo.blocks_of(cols))).astype(np.uint8)
    c, s = B.block8_buffers(rows, cols, "tiles" if tiles else "rows")
    c.view(torch.uint8).copy_(codes.view(torch.uint8))
    s.view(torch.uint8).copy_(torch.from_numpy(e))
    return c, s, bo.decode(codes.view(torch.uint8).numpy(), e)


def _ws(m, n, k):
    """A workspace with no meaning in its bytes (NaN as floats)."""
    return torch.full((B.block8_workspace_bytes(m, n, k),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", MNK)
def test_product_of_whole_numbers_is_exact(m, n, k, kind):
    g = np.random.default_rng(m + n + k)
    for ta, tb, add in ((False, True, False), (False, False, True), (True, True, False), (True, False, True)):
        a, sa, av = _ints(g, m, k, ta)
        b, sb, bv = _ints(g, n, k, tb)
        c = torch.from_numpy(g.integers(-8, 9, (m, n)).astype(F32)).to(DT[kind]).cuda() if add else None
        out = Guarded(m, n, DT[kind])
        B.block8_product(a, sa, b, sb, out.view, add=c, workspace=_ws(m, n, k))
        want = torch.from_numpy(bo.product(av, bv, None if c is None else host(c))).to(DT[kind])
        assert torch.equal(out.view.cpu(), want), (ta, tb, add)
        out.check()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", MNK)
def test_product_of_encoded_values(m, n, k, kind):
    """16-bit outputs: within 2^-10 of the sum of the products' magnitudes (the
    products of neighbouring k are added with 14 bits below the largest: each
    loses less than 2^-13 of it, seven of eight of them) and half a step.  fp32:
    sums of exact products, each addition off by at most a step."""
    g = np.random.default_rng(m * 3 + n + k)
    a, sa, av = device_block8(g.standard_normal((m, k)) * np.exp(g.standard_normal((1, k))))
    b, sb, bv = device_block8(g.standard_normal((n, k)) * 0.1, tiles=True)
    add = torch.from_numpy(g.standard_normal((m, n)).astype(F32)).to(DT[kind]).cuda()
    out = torch.empty(m, n, dtype=DT[kind], device="cuda")
    B.block8_product(a, sa, b, sb, out, add=add, workspace=_ws(m, n, k))
    want = bo.product(av, bv, host(add))
    mag = np.abs(av) @ np.abs(bv).T + np.abs(host(add))
    tol = HALF[kind] * np.abs(want) + LEAST[kind] + mag * (2.0 ** -10 if kind != "f32" else (k + 2) * 2.0 ** -23)
    err = np.abs(host(out) - want)
    assert (err <= tol).all(), float((err / tol).max())
    again = add.clone()  # in place
    B.block8_product(a, sa, b, sb, again, add=again, workspace=_ws(m, n, k))
    assert torch.equal(again, out)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("m,n", [(20, 40), (150, 300)])
def test_product_with_nothing_between_rows_and_with_nan(m, n, kind):
    """Bytes past a row's end are NaN codes and scales, and have no effect; a NaN
    code or scale reaches its own row or column alone."""
    g = np.random.default_rng(2)
    k = 200
    a, sa, av = _ints(g, m, k, False)
    b, sb, bv = _ints(g, n, k, True)
    for t in (a, b):
        t.view(torch.uint8).as_strided((t.shape[0], 8), (t.stride(0), 1), t.storage_offset() + k).fill_(0x7F)
    for t in (sa, sb):
        t.view(torch.uint8).as_strided((t.shape[0], 2), (t.stride(0), 1), t.storage_offset() + 2).fill_(0xFF)
    out = torch.empty(m, n, dtype=DT[kind], device="cuda")
    ws = _ws(m, n, k)
    B.block8_product(a, sa, b, sb, out, workspace=ws)
    want = torch.from_numpy(bo.product(av, bv)).to(DT[kind])
    assert torch.equal(out.cpu(), want)
    a.view(torch.uint8)[3, 199] = 0x7F          # a NaN code
    sa.view(torch.uint8)[7, 0] = 0xFF           # a NaN scale over whole codes
    b.view(torch.uint8)[5, 0] = 0xFF
    B.block8_product(a, sa, b, sb, out, workspace=ws)
    want[3], want[7], want[:, 5] = np.nan, np.nan, np.nan
    assert torch.equal(out.cpu().isnan(), want.isnan())
    assert torch.equal(out.cpu().nan_to_num(0.0), want.nan_to_num(0.0))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [1, 40, 100])
def test_product_over_no_k(m, kind):
    a, sa = B.block8_buffers(m, 0)
    b, sb = B.block8_buffers(24, 0)
    out = torch.full((m, 24), 5.0, dtype=DT[kind], device="cuda")
    add = torch.randn(m, 24, device="cuda").to(DT[kind])
    B.block8_product(a, sa, b, sb, out)
    assert (out == 0).all()
    B.block8_product(a, sa, b, sb, out, add=add)
    assert torch.equal(out, add)
