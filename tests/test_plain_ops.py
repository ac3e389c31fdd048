"""The plain formulations that the GPU tests compare with, pinned on the CPU: gradients by
automatic differentiation and by differences, the mask by its definition, rotations by
complex products."""
import math

import pytest
import torch

from tests import plain_ops as po


def _rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_visible_is_the_definition():
    for nq, nk, w, s in [(5, 9, 3, 2), (7, 7, 1, 0), (4, 4, 9, 9), (1, 6, 2, 1), (3, 8, 0, 0)]:
        see = po.visible(nq, nk, w, s)
        for i in range(nq):
            p = nk - nq + i
            for j in range(nk):
                assert bool(see[i, j]) == (j <= p and (w == 0 or p - j < w or j < s))


def test_attention_equals_library_softmax_attention():
    q, k, v = _rand(2, 9, 16), _rand(2, 9, 16, seed=1), _rand(2, 9, 16, seed=2)
    see = po.visible(9, 9, 4, 1)
    out, lse, *_ = po.attention(q, k, v, see)
    want = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=see)
    assert torch.allclose(out, want, atol=1e-13)
    assert torch.allclose(lse, torch.logsumexp((q @ k.mT / 4).masked_fill(~see, -math.inf), -1))


def _difference(f, x, g, n=6):
    """Central differences of f along n random directions against the gradient g."""
    for s in range(n):
        u, h = _rand(*x.shape, seed=100 + s), 1e-5
        got = float((f(x + h * u) - f(x - h * u)) / (2 * h))
        want = float((g * u).sum())
        assert abs(got - want) <= 1e-6 * max(1.0, abs(want)), (got, want)


@pytest.mark.parametrize("window,sink", [(3, 0), (3, 2), (1, 1), (20, 0)])
def test_attention_gradients(window, sink):
    q, k, v, do = (_rand(11, 8, seed=i) for i in range(4))
    see = po.visible(11, 11, window, sink)
    (dq, _), (dk, _), (dv, _) = po.attention_bwd(q, k, v, do, see)

    def loss(a, b, c):
        z = (a @ b.T * 8 ** -0.5).masked_fill(~see, -math.inf)
        return (torch.softmax(z, -1) @ c * do).sum()

    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    for g, want in zip((dq, dk, dv), torch.autograd.grad(loss(*leaves), leaves)):
        assert torch.allclose(g, want, atol=1e-12)
    _difference(lambda x: loss(x, k, v), q, dq)
    _difference(lambda x: loss(q, x, v), k, dk)
    _difference(lambda x: loss(q, k, x), v, dv)


def _rounded_gradients(q, k, v, do, see, d_factor=1.0):
    """The backward with the kernels' roundings, D taken ``d_factor`` times."""
    r = lambda x: x.bfloat16().double()  # noqa: E731
    scale = q.shape[-1] ** -0.5
    z = (q @ k.mT * scale).masked_fill(~see, -math.inf)
    p = torch.softmax(z, -1)
    out = r(r(p) @ v)
    dz = r(p * (do @ v.mT - d_factor * (do * out).sum(-1, keepdim=True)))
    return r(scale * dz @ k), r(scale * dz.mT @ q), r(r(p).mT @ do)


@pytest.mark.parametrize("n,window,sink", [(300, 300, 0), (300, 100, 4), (200, 2, 1), (500, 60, 130)])
def test_gradients_with_the_kernels_roundings_are_within_their_norms(n, window, sink):
    q, k, v, do = (_rand(2, n, 64, seed=i).bfloat16().double() for i in range(4))
    see = po.visible(n, n, window, sink)
    want = [g for g, _ in po.attention_bwd(q, k, v, do, see)]
    bounds = po.attention_bwd_norms(q, k, v, do, see)
    for got, w, b in zip(_rounded_gradients(q, k, v, do, see), want, bounds):
        assert float((got - w).norm()) <= b <= 0.02 * float(w.norm())
    # What D contributes to dq is not covered when it is off by a tenth.
    off = _rounded_gradients(q, k, v, do, see, 1.1)
    assert float((off[0] - want[0]).norm()) > bounds[0]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 24])
def test_rotation_is_a_complex_product(interleaved, rot):
    x, ang = _rand(5, 24), _rand(5, rot // 2, seed=1)
    y, mag = po.turn(x, ang.cos(), ang.sin(), interleaved)
    z = x[:, :rot].unflatten(1, (rot // 2, 2)) if interleaved else x[:, :rot].unflatten(1, (2, rot // 2)).mT
    t = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(ang), ang)
    t = torch.view_as_real(t)
    want = t.flatten(1) if interleaved else t.mT.flatten(1)
    assert torch.allclose(y[:, :rot], want, atol=1e-13) and torch.equal(y[:, rot:], x[:, rot:])
    assert (mag >= y.abs() - 1e-12).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradients(interleaved):
    x, w, dy, ang = _rand(3, 4, 24), _rand(24, seed=1), _rand(3, 4, 24, seed=2), _rand(3, 4, 8, seed=3)
    c, s = ang.cos(), ang.sin()

    def loss(a, b):
        return (po.norm_rope(a, b, c, s, interleaved, 1e-3)[0] * dy).sum()

    (dx, _), (dw, _) = po.norm_rope_bwd(dy, x, w, c, s, interleaved, 1e-3)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    ga, gb = torch.autograd.grad(loss(a, b), (a, b))
    assert torch.allclose(dx, ga, atol=1e-12) and torch.allclose(dw, gb, atol=1e-12)
    _difference(lambda t: loss(t, w), x, dx)
    _difference(lambda t: loss(x, t), w, dw)
    (g, _), none = po.norm_rope_bwd(dy, x, None, c, s, interleaved, 0.0)
    assert none is None
    a = x.clone().requires_grad_()
    assert torch.allclose(g, torch.autograd.grad((po.norm_rope(a, None, c, s, interleaved, 0)[0] * dy).sum(), a)[0])


def test_gather_pages_follows_the_table():
    pages = torch.arange(4 * 2 * 3 * 1).view(4, 2, 3, 1)
    got = po.gather_pages(pages, torch.tensor([2, 0, 3]), 5)
    assert got[0, :, 0].tolist() == [12, 13, 14, 0, 1] and got[1, :, 0].tolist() == [15, 16, 17, 3, 4]


def test_check_fails_on_a_planted_mistake():
    x = _rand(4, 8)
    po.check("x", x, x, 1e-9 + x.abs() * 0)
    y = x.clone()
    y[1, 2] += 1e-3
    with pytest.raises(AssertionError):
        po.check("x", y, x, 1e-4 + x.abs() * 0)
    y[1, 2] = math.nan
    with pytest.raises(AssertionError):
        po.check("x", y, x, 1e-4 + x.abs() * 0)
