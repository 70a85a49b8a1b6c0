"""The tensor-list operators on the GPU at the ends of their ranges and in
calls that the parity tests do not make: against the oracle where it applies,
with the bounds derived at the head of test_gpu_tensors.py.
"""
import numpy as np
import pytest

from oracle import tensor_oracle as to

from gpu_util import torch_mod
from test_gpu_tensors import Lists, _adam_pair, _same, bits

pytestmark = pytest.mark.gpu

F32 = np.float32


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


@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.5), (0.0, 0.999), (0.9, 0.0)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_largest_gradients_leave_finite_states(kind, beta1, beta2):
    """A finite gradient next to the largest float again and again: no state
    may round to 2^128, which would read as inf and turn 32 weights into NaN."""
    x = Lists([40, 4097], kind, None, True, seed=33, beta1=beta1, beta2=beta2)
    for t in range(10):
        x.step(poison=(1, 70, 3.38e38))
        x.check(t)
    assert all(bool(p.isfinite().all()) for p in x.p)


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_encode_of_the_largest_floats_decodes_finite(rounding):
    torch = torch_mod()
    from zero_partitioned_mixed_buffer_amd import mx8_decode, mx8_encode
    top = 240 * 2.0 ** 120
    vals = np.array([np.finfo(F32).max, -np.finfo(F32).max, 3.2e38, top, -top, 3.1e38, 1e38, 0.0] * 4, dtype=F32)
    x = torch.from_numpy(vals).cuda()
    c, s = torch.zeros(32, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.uint8, device="cuda")
    back = torch.empty(32, device="cuda")
    mx8_encode(x, c, s, rounding=rounding, seed=5)
    mx8_decode(c, s, back)
    want = to.mx8_encode(vals, words=to.random_words(32, 5, 0) if rounding == "stochastic" else None)
    assert np.array_equal(bits(c), want[0]) and int(s) == want[1][0] == 247
    got = back.cpu().numpy()
    assert np.array_equal(got[:5], np.array([top, -top, top, top, -top], dtype=F32))
    assert np.isfinite(got).all() and (np.abs(got - vals)[5:8] <= 2.0 ** 124).all()  # one step of e4m3


# ----------------------------------------------------------------- checkpoints
@pytest.mark.parametrize("src,dst", [(32, 8), (8, 32)])
def test_variance_past_the_range_between_widths(src, dst):
    """A 1e25 gradient leaves a 32-bit list with v = inf and an 8-bit one with
    a root that no 32-bit variance holds; both go on in the other width, and
    the weight moves by less than lr a step: |m| / r is cut to 1, or kept at
    0.1 / sqrt(0.001) = 3.16 (each off by a code, 1/8), and multiplied by 0.9
    sqrt(1-b2^t) / (1-b1^t) < 0.2 at steps 3 and 4."""
    torch = torch_mod()
    a, b = _adam_pair(src)[0], _adam_pair(dst)[0]
    a[2].normal_(0, 1e-3)
    a[0].step()
    a[2][6000] = 1e25
    a[0].step()
    assert a[0].control()["overflow"] == 0 and bool(a[1].isfinite().all())
    b[0].load_state_dict(a[0].state_dict())
    at = b[0].state_offs[2] + 6000 - 5000
    if dst == 32:
        assert float(b[0].exp_avg_sq[at]) == np.finfo(F32).max
        assert bool(b[0].exp_avg.isfinite().all()) and bool(b[0].exp_avg_sq.isfinite().all())
        ratio = float(b[0].exp_avg[at]) / 2.0 ** 64
        assert abs(ratio / (0.1 / 0.001 ** 0.5) - 1) < 0.27  # 9/8 over 8/9
    else:
        assert int((bits(b[0].sq_scale) == 255).sum()) == 0 and int((bits(b[0].avg_scale) == 255).sum()) == 0
    before = b[1].clone()
    b[2].normal_(0, 1e-3)
    b[0].step()
    one = b[1].clone()
    b[0].step()
    torch.cuda.synchronize()
    assert bool(b[1].isfinite().all())
    assert 0 < float((one - before)[6000].abs()) < 1e-3 and 0 < float((b[1] - one)[6000].abs()) < 1e-3
    assert float((b[1] - before).abs().max()) < 2e-2


@pytest.mark.parametrize("state_bits", [8, 32])
def test_checkpoint_of_shaped_tensors(state_bits):
    """Masters and 16-bit copies of different shapes (the list counts elements
    alone): a load restores all of both."""
    torch = torch_mod()
    from zero_partitioned_mixed_buffer_amd import TensorAdam
    torch.manual_seed(2)
    p = [torch.randn(6, 4, device="cuda"), torch.randn((), device="cuda"), torch.randn(3, 1, 70, device="cuda")]
    g = [torch.randn(x.numel(), device="cuda") for x in p]
    w = [x.reshape(shape).bfloat16() for x, shape in zip(p, ((-1,), (1, 1), (7, 30)))]
    a = TensorAdam(p, g, w, state_bits=state_bits, lr=0.1)
    a.step()
    sd = a.state_dict()
    want = [x.clone() for x in p + w]
    for x in p + w:
        x.zero_()
    a.load_state_dict(sd)
    assert all(torch.equal(x, y) for x, y in zip(p + w, want))
    a.step()
    assert not any(torch.equal(x, y) for x, y in zip(p + w, want))


# --------------------------------------------------------------- other streams
@pytest.mark.parametrize("state_bits", [8, 32])
def test_reads_wait_for_steps_on_other_streams(state_bits):
    """Steps given to a side stream, and at once, from the current stream,
    what they left: the control block, the whole state, another step count
    and a load (which no step under way may overwrite)."""
    torch = torch_mod()
    a, b = _adam_pair(state_bits, n=20000001, seed=6)
    x = (torch.randn(a[2].shape, device="cuda") * 1e-3).bfloat16()
    for o in (a, b):
        o[2].copy_(x)
    for _ in range(12):
        b[0].step()
    torch.cuda.synchronize()
    first = a[0].state_dict()
    side = torch.cuda.Stream()

    def steps():
        for _ in range(12):
            a[0].step(stream=side)

    steps()
    got = a[0].state_dict()
    torch.cuda.synchronize()
    want = b[0].state_dict()
    assert set(got) == set(want) and all(np.array_equal(got[k], want[k]) for k in want)
    steps()
    a[0].load_state_dict(first)
    again = a[0].state_dict()
    assert all(np.array_equal(again[k], first[k]) for k in first)
    steps()
    assert a[0].control() == b[0].control()
    steps()
    a[0].set_step(3)
    assert a[0].control()["t"] == 3


def test_shard_reads_wait_for_steps_on_other_streams():
    """The same of the flat window's shard."""
    torch = torch_mod()
    from zero_partitioned_mixed_buffer_amd import OwnedShard
    n, nd = 8000000, 4
    p0 = torch.randn(n, device="cuda") * 0.02
    a, b = (OwnedShard(p0, loss_scale=1.0) for _ in range(2))
    slices = (torch.randn(nd, n, device="cuda") * 1e-3).half()
    ag = torch.zeros(n, dtype=torch.float16, device="cuda")
    for _ in range(12):
        b.step(slices, allgather=ag)
    torch.cuda.synchronize()
    first = a.state_dict()
    side = torch.cuda.Stream()

    def steps():
        for _ in range(12):
            a.step(slices, allgather=ag, stream=side)

    steps()
    got = a.state_dict()
    torch.cuda.synchronize()
    want = b.state_dict()
    assert all(np.array_equal(got[k], want[k]) for k in want)
    steps()
    a.load_state_dict(first)
    again = a.state_dict()
    assert all(np.array_equal(again[k], first[k]) for k in ("master", "exp_avg", "exp_avg_sq"))
    steps()
    assert a.control()["t"] == 12


@pytest.mark.parametrize("state_bits", [8, 32])
def test_first_step_on_another_stream(state_bits):
    """Made while its stream still has work to do, and stepped at once on
    another one: the states and tables are there."""
    torch = torch_mod()
    from zero_partitioned_mixed_buffer_amd import OwnedShard, TensorAdam
    n = 3000001
    p0 = torch.randn(n, device="cuda") * 0.02
    g = (torch.randn(n, device="cuda") * 1e-3).half()
    slices = g.view(1, n)
    busy = torch.zeros(1 << 30, device="cuda")
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side):
        p, ag = p0.clone(), torch.zeros(n, dtype=torch.float16, device="cuda")
        torch.cuda.synchronize()
        for _ in range(20):  # about 30 ms
            busy.add_(1.0)
        opt = TensorAdam([p], [g], state_bits=state_bits, seed=8)
        opt.step(stream=stream)
        for _ in range(20):
            busy.add_(1.0)
        shard = OwnedShard(p0, loss_scale=1.0)
        shard.step(slices, allgather=ag, stream=stream)
        torch.cuda.synchronize()
        assert opt.control()["t"] == shard.control()["t"] == 1
        got.append([p, ag, opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8), *shard.committed()])
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_checkpoint_brings_the_random_words(rounding, tmp_path):
    """A list of another seed, rounding and offsets goes on exactly as the one
    that was saved."""
    torch = torch_mod()
    other = "stochastic" if rounding == "nearest" else "nearest"
    a = _adam_pair(8, seed=2 ** 64 - 3, rounding=rounding, flat_offs=[5, 2 ** 40, 7])[0]
    b = _adam_pair(8, seed=78, rounding=other)[0]
    c = _adam_pair(8, seed=79, rounding=rounding, flat_offs=[0, 33, 5000])[0]
    x = (torch.randn(a[2].shape, device="cuda") * 1e-3).bfloat16()
    for o in (a, b, c):
        o[2].copy_(x)
    a[0].step()
    a[0].save(str(tmp_path / "s.npz"))
    b[0].load(str(tmp_path / "s.npz"))
    c[0].load_state_dict(a[0].state_dict())
    assert b[0].rounding == rounding and b[0].seed == 2 ** 64 - 3 and b[0].flat_offs == [5, 2 ** 40, 7]
    for t in range(2):
        for o in (a, b, c):
            o[0].step()
        torch.cuda.synchronize()
        _same(a, b)
        _same(a, c)
    b[0].set_grads([g.clone() for g in b[0].grads])  # the offsets stay
    for o in (a, b):
        o[0].step()
    torch.cuda.synchronize()
    _same(a, b)


def test_checkpoint_refusals_leave_the_list_as_it_was():
    torch = torch_mod()
    from zero_partitioned_mixed_buffer_amd import binding as B
    a, b = _adam_pair(8, seed=3), _adam_pair(8, seed=4)
    a, b, c = a[0], b[0], b[1]
    a[2].normal_(0, 1e-3)
    a[0].step()
    sd = a[0].state_dict()
    for bad, kind in ((dict(rounding=np.asarray("up")), ValueError), (dict(flat_offs=np.array([0, 1])), ValueError),
                      (dict(flat_offs=np.array([0, 33, -1])), B.ZeroError), (dict(exp_avg=sd["exp_avg"][1:]), ValueError),
                      (dict(ctl=sd["ctl"][1:]), ValueError)):
        with pytest.raises(kind):
            b[0].load_state_dict({**sd, **bad})
        torch.cuda.synchronize()
        _same(b, c)
        assert b[0].seed == 4 and b[0].rounding == "stochastic"
    # a state_dict without the words' parameters: the list keeps its own
    b[0].load_state_dict({k: v for k, v in sd.items() if k not in ("seed", "rounding", "flat_offs")})
    _same(a, b)
    assert b[0].seed == 4


# -------------------------------------------------------------------- autograd
@pytest.mark.parametrize("state_bits", [8, 32])
def test_backward_through_a_step_raises(state_bits):
    """A graph that saved a weight or its 16-bit copy before a step refuses
    its backward pass, as after torch's own in-place operations; one made
    after it runs."""
    torch = torch_mod()
    from zero_partitioned_mixed_buffer_amd import TensorAdam, binding as B
    torch.manual_seed(4)
    p = torch.nn.Parameter(torch.randn(40, 5, device="cuda"))
    w = torch.nn.Parameter(p.detach().bfloat16())
    p.grad = torch.randn_like(p)
    opt = TensorAdam([p], [p.grad], [w], state_bits=state_bits)
    for x in (p, w):
        y = (x * x).sum()
        opt.step()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    lst = opt.list
    y = (p * p).sum()
    B.tensors_adam_step(lst, opt.hp, opt.ctl, opt.workspace)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    w.grad = None
    (w * w).sum().backward()
    assert torch.equal(w.grad, 2 * w.detach())
    # tensors that no graph knows are not counted
    q = torch.randn(100, device="cuda")
    plain = TensorAdam([q], [torch.randn(100, device="cuda")], state_bits=state_bits)
    at = q._version
    plain.step()
    assert q._version == at and not plain.list.written


@pytest.mark.parametrize("state_bits", [8, 32])
def test_gradients_made_anew_each_step(state_bits):
    """A loop with zero_grad()'s default: autograd's new gradients, named by
    set_grads, step as the same values copied into the first ones do."""
    torch = torch_mod()
    from zero_partitioned_mixed_buffer_amd import TensorAdam
    torch.manual_seed(1)
    net = torch.nn.Sequential(torch.nn.Linear(33, 70), torch.nn.Tanh(), torch.nn.Linear(70, 5)).cuda()
    params = list(net.parameters())
    twins = [p.detach().clone() for p in params]
    held = [torch.zeros_like(p) for p in twins]
    for p in params:
        p.grad = torch.zeros_like(p)
    a = TensorAdam(params, [p.grad for p in params], state_bits=state_bits, seed=3)
    b = TensorAdam(twins, held, state_bits=state_bits, seed=3)
    keep = [p.grad for p in params]  # so that no new gradient can take an old one's place
    for t in range(4):
        net.zero_grad()
        net(torch.randn(64, 33, device="cuda")).square().mean().backward()
        assert all(p.grad.data_ptr() != g.data_ptr() for p, g in zip(params, keep))
        a.set_grads([p.grad for p in params])
        keep = [p.grad for p in params]
        for h, p in zip(held, params):
            h.copy_(p.grad)
        a.step()
        b.step()
        torch.cuda.synchronize()
        assert all(torch.equal(p.detach(), q) for p, q in zip(params, twins))
        assert a.control() == b.control() and a.control()["t"] == t + 1
