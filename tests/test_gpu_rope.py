"""Per-head norms with the rotation, forward and backward, against the float64 formulas,
value by value (tests/plain_ops.py derives the bounds)."""
import pytest
import torch

from tests import plain_ops as po

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _moba():
    import block_sparse_long_prefill_b200 as moba
    return moba


def _table(positions, rot):
    f = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return a.cos().float(), a.sin().float()


def _case(batch, hq, hkv, n, d, rot, norm, given, seed=0, strided=True):
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if strided:
        x = rand(batch, n, hq + hkv, d).bfloat16().permute(0, 2, 1, 3)
        q, k = x[:, :hq], x[:, hq:]
    else:
        q, k = rand(batch, hq, n, d).bfloat16(), rand(batch, hkv, n, d).bfloat16()
    cos, sin = _table(n + 50, rot)
    pos = torch.randint(0, n + 50, (batch, n), generator=g, device="cuda", dtype=torch.int32) if given else None
    w = {"none": (None, None), "bf16": ((1 + 0.3 * rand(d)).bfloat16(), (1 + 0.3 * rand(d)).bfloat16()),
         "f32": (1 + 0.3 * rand(d), 1 + 0.3 * rand(d)), "q": (1 + 0.3 * rand(d), None)}[norm]
    at = torch.arange(n, device="cuda").expand(batch, n) if pos is None else pos.long()
    return q, k, cos, sin, pos, w, (cos.double()[at][:, None], sin.double()[at][:, None]), rand


CASES = [
    # batch, hq, hkv, n, d, rot, norm, given, interleaved
    (1, 1, 1, 1, 64, 64, "bf16", False, False),
    (2, 5, 3, 7, 64, 16, "none", True, False),
    (1, 9, 1, 130, 64, 48, "f32", True, True),
    (3, 4, 2, 33, 80, 80, "bf16", False, False),
    (1, 3, 3, 101, 80, 32, "q", True, True),
    (2, 2, 1, 2, 80, 64, "none", False, True),
    (1, 8, 2, 257, 128, 128, "bf16", True, False),
    (2, 6, 2, 65, 128, 64, "f32", False, True),
    (1, 32, 8, 700, 128, 112, "none", True, False),
]


@pytest.mark.parametrize("batch,hq,hkv,n,d,rot,norm,given,inter", CASES)
def test_forward(batch, hq, hkv, n, d, rot, norm, given, inter):
    moba = _moba()
    q, k, cos, sin, pos, w, (c, s), _ = _case(batch, hq, hkv, n, d, rot, norm, given, seed=n)
    qo, ko = moba.qk_norm_rope_fwd(q, k, cos, sin, pos, w[0], w[1], EPS, inter)
    assert moba.device_status() == 0
    for name, x, y, wt in (("q", q, qo, w[0]), ("k", k, ko, w[1])):
        po.check(name, y, *po.norm_rope(x.double(), None if wt is None else wt.double(), c, s, inter, EPS))


@pytest.mark.parametrize("batch,hq,hkv,n,d,rot,norm,given,inter", CASES)
def test_backward(batch, hq, hkv, n, d, rot, norm, given, inter):
    moba = _moba()
    q, k, cos, sin, pos, w, (c, s), rand = _case(batch, hq, hkv, n, d, rot, norm, given, seed=n + 1)
    gq, gk = rand(batch, hq, n, d).bfloat16(), rand(batch, hkv, n, d).bfloat16()
    got = moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, w[0], w[1], EPS, inter)
    again = moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, w[0], w[1], EPS, inter)
    assert moba.device_status() == 0
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)
    for name, g, x, dx, wt, dw in (("q", gq, q, got[0], w[0], got[2]), ("k", gk, k, got[1], w[1], got[3])):
        want, wdw = po.norm_rope_bwd(g.double(), x.double(), None if wt is None else wt.double(), c, s, inter, EPS)
        po.check("d" + name, dx, *want)
        if wt is None:
            assert dw is None
        else:
            po.check("dw" + name, dw, *wdw)


def test_in_place_equals_out_of_place():
    moba = _moba()
    for d in (64, 80, 128):
        q, k, cos, sin, pos, w, _, rand = _case(2, 6, 3, 77, d, 32, "bf16", True, seed=d)
        want = moba.qk_norm_rope_fwd(q, k, cos, sin, pos, *w, EPS)
        qi, ki = q.clone(), k.clone()
        moba.qk_norm_rope_fwd(qi, ki, cos, sin, pos, *w, EPS, q_out=qi, k_out=ki)
        assert torch.equal(qi, want[0]) and torch.equal(ki, want[1])
        gq, gk = rand(*q.shape).bfloat16(), rand(*k.shape).bfloat16()
        want = moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, *w, EPS)
        moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, *w, EPS, dq=gq, dk=gk)
        assert torch.equal(gq, want[0]) and torch.equal(gk, want[1])


def test_large_and_tiny_rows_and_zero_rows():
    """Rows of 2^+-60 keep their norm in float32 (their squares 2^+-120), zero rows give
    zeros, infinities outside the rotation pass."""
    moba = _moba()
    q, k, cos, sin, pos, w, (c, s), _ = _case(1, 4, 1, 9, 128, 64, "bf16", False, strided=False)
    q[:, 0] *= 2.0 ** 60
    q[:, 1] *= 2.0 ** -30
    q[:, 2] = 0
    qo, ko = moba.qk_norm_rope_fwd(q, k, cos, sin, None, *w, EPS)
    po.check("q", qo, *po.norm_rope(q.double(), w[0].double(), c, s, False, EPS))
    assert not qo[:, 2].any()
    k[..., 100] = float("inf")
    for inter in (False, True):
        _, ko = moba.qk_norm_rope_fwd(q, k, cos, sin, interleaved=inter)
        assert torch.isinf(ko[..., 100]).all() and torch.isfinite(ko[..., :100]).all()
        assert torch.equal(ko[..., 101:], k[..., 101:])


def test_positions_outside_the_table_are_left_out():
    moba = _moba()
    q, k, cos, sin, pos, w, (c, s), rand = _case(1, 3, 1, 20, 64, 64, "f32", True)
    good = pos.clone()
    pos[0, 3], pos[0, 11] = -1, cos.shape[0]
    qo, ko = torch.full(q.shape, 7.0, device="cuda").bfloat16(), torch.full(k.shape, 7.0, device="cuda").bfloat16()
    moba.qk_norm_rope_fwd(q, k, cos, sin, pos, *w, EPS, q_out=qo, k_out=ko)
    assert moba.device_status() == -10 and moba.device_status() == 0
    want, _ = moba.qk_norm_rope_fwd(q, k, cos, sin, good, *w, EPS)
    rows = [i for i in range(20) if i not in (3, 11)]
    assert torch.equal(qo[:, :, rows], want[:, :, rows])
    assert (qo[:, :, [3, 11]] == 7).all() and (ko[:, :, [3, 11]] == 7).all()
    # The backward leaves these rows out of the weights' gradients too.
    gq, gk = rand(*q.shape).bfloat16(), rand(*k.shape).bfloat16()
    got = moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, *w, EPS)
    assert moba.device_status() == -10
    at = good.clone()
    gq[:, :, [3, 11]] = 0
    gk[:, :, [3, 11]] = 0
    want = moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, at, *w, EPS)
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])


@pytest.mark.parametrize("d", [64, 80, 128])
def test_without_an_epsilon(d):
    """eps = 0 is allowed; lanes without a row (n no multiple of a warp's rows, positions out of
    range) must not leave 0 / 0 in the weights' gradients."""
    moba = _moba()
    q, k, cos, sin, pos, w, (c, s), rand = _case(2, 3, 1, 13, d, 32, "f32", True, seed=d)
    gq, gk = rand(*q.shape).bfloat16(), rand(*k.shape).bfloat16()
    qo, ko = moba.qk_norm_rope_fwd(q, k, cos, sin, pos, *w, 0.0)
    po.check("q", qo, *po.norm_rope(q.double(), w[0].double(), c, s, False, 0.0))
    got = moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, *w, 0.0)
    for name, g, x, dx, wt, dw in (("q", gq, q, got[0], w[0], got[2]), ("k", gk, k, got[1], w[1], got[3])):
        want, wdw = po.norm_rope_bwd(g.double(), x.double(), wt.double(), c, s, False, 0.0)
        po.check("d" + name, dx, *want)
        po.check("dw" + name, dw, *wdw)
    pos[0, 5] = -1
    got = moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, *w, 0.0)
    assert moba.device_status() == -10
    assert torch.isfinite(got[2]).all() and torch.isfinite(got[3]).all()


def test_in_a_graph_and_on_another_stream():
    moba = _moba()
    q, k, cos, sin, pos, w, _, rand = _case(1, 8, 2, 300, 128, 128, "bf16", True)
    gq, gk = rand(*q.shape).bfloat16(), rand(*k.shape).bfloat16()
    want = (*moba.qk_norm_rope_fwd(q, k, cos, sin, pos, *w, EPS),
            *moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, *w, EPS))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*moba.qk_norm_rope_fwd(q, k, cos, sin, pos, *w, EPS, stream=side),
           *moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, *w, EPS, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*moba.qk_norm_rope_fwd(q, k, cos, sin, pos, *w, EPS),
               *moba.qk_norm_rope_bwd(gq, gk, q, k, cos, sin, pos, *w, EPS))
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
