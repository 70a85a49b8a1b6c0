"""The 8-bit layer operators on columns of one buffer (GPU): inputs and outputs
side by side in the same rows, in either order, give what buffers of their own do."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
B = pytest.importorskip("zero_partitioned_mixed_buffer_amd.binding")

ORDERS = [(0, 1, 2), (2, 1, 0), (1, 2, 0), (0, 2, 1)]


def columns(matrices, order, gap=3):
    """Copies of matrices [rows, c] in one buffer, `gap` columns around each, in
    the given order: (views, a check that the rest was left alone)."""
    rows, dtype = matrices[0].shape[0], matrices[0].dtype
    width = gap + sum(m.shape[1] + gap for m in matrices)
    box = torch.full((rows, width), 99.0, dtype=dtype, device="cuda")
    views, at = [None] * len(matrices), gap
    for i in order:
        views[i] = box[:, at:at + matrices[i].shape[1]]
        views[i].copy_(matrices[i])
        at += matrices[i].shape[1] + gap
    untouched = torch.ones_like(box, dtype=torch.bool)
    for v in views:
        at = v.storage_offset()
        untouched[:, at:at + v.shape[1]] = False
    return views, lambda: bool((box[untouched] == 99).all())


def same_codes(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("rows,cols", [(1, 40), (130, 300), (70, 2049), (9, 20001)])
def test_norm_and_gradients(rows, cols, order):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, r, dh = (torch.randn(rows, cols, generator=g, device="cuda").bfloat16() for _ in range(3))
    w = torch.randn(cols, generator=g, device="cuda")

    def forward(x, r, h):
        (c, s), rstd = B.block8_buffers(rows, cols), torch.empty(rows, device="cuda")
        B.rms_norm8(x, w, c, s, rstd, residual=r, h=h)
        return c, s, rstd

    h = torch.empty_like(x)
    c, s, rstd = forward(x, r, h)
    views, rest = columns([x, r, torch.zeros_like(x)], order)
    c2, s2, rstd2 = forward(*views)
    assert torch.equal(views[2], h) and torch.equal(rstd2, rstd) and same_codes(c2, c) and same_codes(s2, s) and rest()
    assert torch.equal(views[0], x) and torch.equal(views[1], r)

    ws = torch.empty(B.rms_norm8_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")

    def backward(dy, h, dx, dh=None):
        dw = torch.empty(cols, device="cuda")
        B.rms_norm8_backward(dy, h, w, rstd, dx, dw, ws, dh=dh)
        return dw

    dx = torch.empty_like(x)
    dw = backward(x, h, dx, dh)
    views, rest = columns([x, h, torch.zeros_like(x)], order)
    assert torch.equal(backward(*views, dh=dh), dw) and torch.equal(views[2], dx) and rest()
    assert torch.equal(views[0], x) and torch.equal(views[1], h)


@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
@pytest.mark.parametrize("m,n,k", [(20, 30, 200), (300, 200, 9000), (2300, 800, 200), (2900, 2900, 200)])
def test_product_beside_its_addend(m, n, k, order):
    g = torch.Generator(device="cuda").manual_seed(m)
    a, b = B.block8_buffers(m, k), B.block8_buffers(n, k)
    B.block8_encode(torch.randn(m, k, generator=g, device="cuda"), *a)
    B.block8_encode(torch.randn(n, k, generator=g, device="cuda"), *b)
    add = torch.randn(m, n, generator=g, device="cuda")
    ws = torch.empty(B.block8_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(add)
    B.block8_product(*a, *b, out, add=add, workspace=ws)
    views, rest = columns([add, torch.zeros_like(add)], order)
    B.block8_product(*a, *b, views[1], add=views[0], workspace=ws)
    assert torch.equal(views[1], out) and torch.equal(views[0], add) and rest()


@pytest.mark.parametrize("blocks", ["rows", "tiles"])
def test_codes_in_one_buffer(blocks):
    """Codes of several layers' matrices in the columns of one buffer."""
    g = torch.Generator(device="cuda").manual_seed(7)
    shapes = [(200, 300), (200, 130), (200, 600)]
    box = torch.full((200, 1200), 0x55, dtype=torch.uint8, device="cuda")
    at, untouched = 16, torch.ones_like(box, dtype=torch.bool)
    views = []
    for rows, cols in shapes:
        views.append(box[:, at:at + cols].view(torch.float8_e4m3fn))
        untouched[:, at:at + cols] = False
        at += (cols + 31) // 16 * 16
    for view, (rows, cols) in zip(views, shapes):
        x = torch.randn(rows, cols, generator=g, device="cuda")
        c, s = B.block8_buffers(rows, cols, blocks)
        _, s2 = B.block8_buffers(rows, cols, blocks)
        B.block8_encode(x, c, s, blocks=blocks)
        B.block8_encode(x, view, s2, blocks=blocks)
        assert same_codes(view, c) and same_codes(s2, s)
    assert bool((box[untouched] == 0x55).all())
