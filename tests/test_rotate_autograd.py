"""rotate under autograd: the result's gradient, what is refused, and what has to stay as it
is.  On the CPU the library's call is replaced by the definition in 64 bits."""
import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests import page_ref as R

BF, HF = torch.bfloat16, torch.float16
NEW, ROWS = [1, 13, 0, 5], [1, 40, 9, 3000]


def _positions(b):
    cu, m = b["cu_q"].tolist(), b["kv_len"].tolist()
    return [(cu[r], cu[r + 1], torch.arange(m[r] - cu[r + 1] + cu[r], m[r]))
            for r in range(b["num_req"])]


def _definition(b, x, rope, pos, inverse, out, d_err, stream=None):
    runs = [(0, b["num_q"], pos)] if pos is not None else _positions(b)
    for lo, hi, p in runs:
        out.data[lo:hi] = R.rotate(x.detach()[lo:hi], p, rope, inverse).to(x.dtype)
    return S.OK


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def dev(request, monkeypatch):
    if request.param == "cpu":
        monkeypatch.setattr(S, "csa2_rotate", _definition)
    return request.param


def _normal(shape, dtype, dev, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(dev)


def _rope(dev, rot=32, interleaved=False, amplitude=1.25):
    return dict(S.rope_freqs(rot, scaling="linear", factor=2, device=dev), interleaved=interleaved,
                amplitude=amplitude)


def _garbage(dev):
    """Memory that a fresh tensor may get: not zeros."""
    for n in (1 << 12, 1 << 14, 1 << 16, 1 << 18):
        torch.full((n,), float("nan"), dtype=BF, device=dev)


@pytest.mark.parametrize("interleaved,dtype,given", [(False, BF, False), (True, HF, False),
                                                     (False, HF, True)])
def test_gradient_is_the_rotation_turned_round(dev, interleaved, dtype, given):
    b, cu = R.batch(NEW, ROWS, dev, lead=3, tail=2)
    rope = _rope(dev, interleaved=interleaved)
    pos = torch.arange(b["num_q"], device=dev) * 7 if given else None
    x = _normal((b["num_q"] + 4, 3, 64), dtype, dev).requires_grad_()
    _garbage(dev)
    y = S.rotate(b, x, rope, pos=pos)
    g = _normal(x.shape, dtype, dev, 1)
    _garbage(dev)
    got, = torch.autograd.grad(y, x, g)
    with torch.no_grad():
        fwd = S.rotate(b, x, rope, pos=pos)
        back = S.rotate(b, g, rope, pos=pos, inverse=True)
    mine = slice(0, b["num_q"]) if given else slice(cu[0], cu[-1])
    assert torch.equal(y[mine], fwd[mine]) and torch.equal(got[mine], back[mine])
    other = torch.ones(x.shape[0], dtype=torch.bool)
    other[mine] = False
    assert (y[other.to(dev)] == 0).all() and (got[other.to(dev)] == 0).all()
    assert not fwd.requires_grad


def test_gradient_by_differences(dev):
    """d/dt sum(c * rotate(x + t e)) at 0, the call being linear: the difference of two calls
    is the gradient along e, but for roundings of half a step of each value."""
    b, _ = R.batch([9], [86], dev)
    rope = _rope(dev)
    x = _normal((9, 2, 64), HF, dev, 1).requires_grad_()
    c, e = _normal(x.shape, HF, dev, 2), _normal(x.shape, HF, dev, 3)
    (S.rotate(b, x, rope).double() * c.double()).sum().backward()
    with torch.no_grad():
        p, m = x + e, x - e
        up, down = S.rotate(b, p, rope).double(), S.rotate(b, m, rope).double()
        step = (p.double() - m.double()) / 2
    want = ((up - down) / 2 * c.double()).sum()
    got = (x.grad.double() * step).sum()
    tol = 2.0 ** -11 * ((up.abs() + down.abs()) / 2 * c.double().abs()).sum() \
        + 2.0 ** -11 * (x.grad.double().abs() * step.abs()).sum() \
        + 2.0 ** -18 * 1.25 * 2 * (p.double().abs() + m.double().abs()).sum() * c.double().abs().max()
    assert (got - want).abs() <= tol
    assert tol < 0.02 * (x.grad.double().abs() * step.abs()).sum()


def test_through_a_projection_and_of_second_order(dev):
    """Weights in front of the rotation get their gradient; a gradient that requires one."""
    b, _ = R.batch([6], [50], dev)
    rope = _rope(dev, amplitude=1.0)
    w = _normal((16, 2 * 64), BF, dev, 4).requires_grad_()
    h = _normal((6, 16), BF, dev, 5)
    y = S.rotate(b, (h @ w).view(6, 2, 64), rope)
    s = y.float().square().sum() / 2
    s.backward()
    # a rotation keeps the length of what it turns: the gradient is that without it, but for
    # three roundings (rotated, its gradient, the product) and those of the projection
    p = h.double() @ w.detach().double()
    want = h.double().t() @ p
    tol = h.double().abs().t() @ (p.abs() + p.abs().amax(1, keepdim=True)) * 2.0 ** -8 * 8
    assert ((w.grad.double() - want).abs() <= tol).all()

    x = _normal((6, 2, 64), HF, dev, 6).requires_grad_()
    y = S.rotate(b, x, rope)
    v = _normal(x.shape, HF, dev, 7).requires_grad_()
    g, = torch.autograd.grad(y, x, v, create_graph=True)
    gg, = torch.autograd.grad(g, v, torch.ones_like(g))
    with torch.no_grad():
        assert torch.equal(gg, S.rotate(b, torch.ones_like(x), rope))


def test_gradients_as_they_come(dev):
    """Ones that are expanded, transposed or off their alignment; the same leaf twice."""
    b, _ = R.batch([5], [5], dev)
    rope = _rope(dev)
    x = _normal((5, 4, 64), HF, dev, 8).requires_grad_()
    with torch.no_grad():
        want = S.rotate(b, torch.ones_like(x), rope, inverse=True)
    S.rotate(b, x, rope).sum().backward()
    assert torch.equal(x.grad, want)
    ones = torch.ones((4, 64, 5), dtype=HF, device=dev).permute(2, 0, 1)
    off = torch.ones(x.numel() + 1, dtype=HF, device=dev)[1:].view(x.shape)
    for g in (ones, off):
        got, = torch.autograd.grad(S.rotate(b, x, rope), x, g)
        assert torch.equal(got, want)
    x.grad = None
    (S.rotate(b, x, rope) + S.rotate(b, x, rope, inverse=True)).sum().backward()
    with torch.no_grad():
        both = want + S.rotate(b, torch.ones_like(x), rope)
    assert torch.equal(x.grad, both)


def test_refusals(dev):
    b, _ = R.batch([5], [5], dev)
    rope = _rope(dev)
    x = _normal((5, 4, 64), HF, dev, 9)
    leaf = x.clone().requires_grad_()
    for args in ((leaf, leaf), (leaf, torch.empty_like(x)), (x, leaf)):
        with pytest.raises(S.Csa2Error, match="out="):
            S.rotate(b, args[0], rope, out=args[1])
    hot = dict(rope, freq=rope["freq"].clone().requires_grad_())
    with pytest.raises(S.Csa2Error, match="frequencies"):
        S.rotate(b, x, hot)
    with torch.no_grad():                # as in a server whose weights require gradients
        want = S.rotate(b, x, rope)
        assert torch.equal(S.rotate(b, leaf, hot, out=leaf), want)
    assert not S.rotate(b, x, rope).requires_grad


def test_what_was_saved_has_to_stay(dev):
    """A batch whose lengths go on, and rows that are turned where they lie, are noticed."""
    b, _ = R.batch([5], [5], dev)
    rope = _rope(dev)
    x = _normal((5, 4, 64), HF, dev, 10)
    leaf = x.clone().requires_grad_()
    y = S.rotate(b, leaf, rope)
    b["kv_len"] += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    s = (leaf * x).sum()                 # saves x
    S.rotate(b, x, rope, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        s.backward()


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph():
    dev = "cuda"
    b, _ = R.batch([300], [300], dev)
    rope = _rope(dev, 64)
    x = _normal((300, 16, 64), HF, dev, 11).requires_grad_()
    g = _normal(x.shape, HF, dev, 12)
    y = S.rotate(b, x, rope)
    want, = torch.autograd.grad(y, x, g)
    keep = y.detach().clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        y = S.rotate(b, x, rope, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        got, = torch.autograd.grad(y, x, g)
        assert torch.equal(y, keep) and torch.equal(got, want)
        del y, got
    # one graph with the gradient, no eager graph of the same leaf alive
    xs, gs = x.detach().clone().requires_grad_(), g.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = S.rotate(b, xs, rope)
        got, = torch.autograd.grad(y, xs, gs)
    for sign in (1, -1):
        with torch.no_grad():
            xs.copy_(x * sign), gs.copy_(g * sign)
        graph.replay()
        assert torch.equal(y, keep * sign) and torch.equal(got, want * sign)
