"""Sliding-window attention with sinks and its backward against the float64 formulas, value
by value within what the roundings allow (tests/plain_ops.py derives the bounds)."""
import pytest
import torch

from tests import plain_ops as po

pytestmark = pytest.mark.gpu


def _moba():
    import block_sparse_long_prefill_b200 as moba
    return moba


def _inputs(batch, hq, hkv, n, nk, d, seed, strided=False):
    g = torch.Generator("cuda").manual_seed(seed)

    def rand(h, m):
        if strided:  # token-major: the heads of a token lie side by side
            return torch.randn(batch, m, h, d, generator=g, device="cuda").bfloat16().permute(0, 2, 1, 3)
        return torch.randn(batch, h, m, d, generator=g, device="cuda").bfloat16()

    return rand(hq, n), rand(hkv, nk), rand(hkv, nk), rand(hq, n)


def _wide(x, G):
    return x.double().repeat_interleave(G, 1)


def _fwd(batch, hq, hkv, n, nk, d, window, sink, seed=0, strided=False, scale=0.0):
    moba = _moba()
    q, k, v, do = _inputs(batch, hq, hkv, n, nk, d, seed, strided)
    out, lse = moba.swa_attn_fwd_chunk(q, k, v, window, scale, sink=sink)
    assert moba.device_status() == 0
    see = po.visible(n, nk, window, sink, "cuda")
    G = hq // hkv
    o, l, p, ob, lb = po.attention(q.double(), _wide(k, G), _wide(v, G), see, scale or None)
    po.check("out", out, o, ob)
    po.check("lse", lse, l, lb)
    return (q, k, v, do), (out, lse), see, ob


def _bwd(batch, hq, hkv, n, d, window, sink, seed=0, strided=False, scale=0.0):
    moba = _moba()
    (q, k, v, do), (out, lse), see, ob = _fwd(batch, hq, hkv, n, n, d, window, sink, seed, strided, scale)
    dq, dk, dv = moba.swa_attn_bwd(q, k, v, out, lse, do, window, sink, scale)
    assert moba.device_status() == 0
    G = hq // hkv
    (wq, bq), (wk, bk), (wv, bv) = po.attention_bwd(q.double(), _wide(k, G), _wide(v, G), do.double(), see,
                                                    scale or None, ob)
    fold = lambda x: x.view(batch, hkv, G, n, d).sum(2)  # noqa: E731
    po.check("dq", dq, wq, bq)
    # Stored after the sum over the heads: the heads' own bounds cover its rounding.
    po.check("dk", dk, fold(wk), fold(bk))
    po.check("dv", dv, fold(wv), fold(bv))
    return (q, k, v, do, out, lse), (dq, dk, dv)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("n,window,sink", [(1, 1, 1), (5, 2, 1), (129, 1, 128), (257, 64, 4), (640, 128, 129),
                                           (1000, 200, 4), (1000, 5000, 4), (777, 100, 2000), (1100, 130, 300)])
def test_forward(d, n, window, sink):
    _fwd(1, 2, 2, n, n, d, window, sink, seed=n)


@pytest.mark.parametrize("d,hq,hkv,n,nk,window,sink", [
    (64, 3, 1, 100, 1000, 77, 4), (80, 4, 2, 1, 1500, 300, 130), (128, 8, 2, 333, 900, 128, 1),
    (128, 2, 2, 130, 131, 3, 2)])
def test_forward_of_the_last_rows(d, hq, hkv, n, nk, window, sink):
    _fwd(2, hq, hkv, n, nk, d, window, sink, seed=nk, strided=True)


def test_forward_without_sinks_is_the_band():
    moba = _moba()
    q, k, v, _ = _inputs(1, 4, 2, 900, 900, 128, 3)
    a, la = moba.swa_attn_fwd(q, k, v, 200)
    b, lb = moba.swa_attn_fwd(q, k, v, 200, sink=0)
    assert torch.equal(a, b) and torch.equal(la, lb)
    # Sinks inside every row's window change nothing that is seen (the sums run in another
    # order: within the bounds, not to the bit).
    _fwd(1, 4, 2, 150, 150, 128, 200, 9)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("n,window,sink", [(1, 1, 0), (5, 2, 1), (128, 128, 0), (129, 1, 128), (257, 64, 4),
                                           (640, 128, 129), (1000, 200, 4), (1000, 5000, 4), (900, 100, 2000)])
def test_backward(d, n, window, sink):
    _bwd(1, 2, 2, n, d, window, sink, seed=n)


@pytest.mark.parametrize("d,batch,hq,hkv,n,window,sink", [
    (64, 2, 6, 2, 500, 130, 5), (80, 2, 4, 1, 700, 60, 140), (128, 2, 8, 4, 520, 128, 130),
    (128, 1, 3, 1, 3000, 1, 1), (64, 1, 8, 1, 3000, 100, 260), (80, 1, 1, 1, 2900, 250, 0)])
def test_backward_of_shared_heads_and_split_sinks(d, batch, hq, hkv, n, window, sink):
    _bwd(batch, hq, hkv, n, d, window, sink, seed=n, strided=True)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("window,sink", [(1, 1), (40, 0), (300, 4), (2000, 150)])
def test_several_items_a_block(d, window, sink):
    """More query and key tiles than the GPU has SMs, of walks of one chunk and of many: a
    block's next item starts while its last one is read out."""
    _bwd(2, 16, 4, 1100, d, window, sink, seed=window)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("up", [True, False])
def test_scores_that_climb_or_fall_by_hundreds(d, up):
    """Keys whose scores rise along the sequence raise the running maximum in every chunk (by
    far more than 2^8), and falling ones never; probabilities reach one key or many."""
    moba = _moba()
    n, window, sink = 1300, 500, 70
    q, k, v, do = _inputs(1, 2, 1, n, n, d, 21)
    ramp = torch.linspace(0, 1, n, device="cuda")
    ramp = ramp if up else 1 - ramp
    # One direction carries the ramp: 8 x 8 x 60 x d^-0.5, 480 natural units at d = 64.
    q[..., 0] = 8.0
    k[..., 0] = (480 * ramp).bfloat16()
    out, lse = moba.swa_attn_fwd(q, k, v, window, sink=sink)
    dq, dk, dv = moba.swa_attn_bwd(q, k, v, out, lse, do, window, sink)
    assert moba.device_status() == 0
    see = po.visible(n, n, window, sink, "cuda")
    o, l, p, ob, lb = po.attention(q.double(), _wide(k, 2), _wide(v, 2), see)
    # Scores of hundreds carry float32 errors of their own size: (d + 8) 2^-24 of the sum of
    # magnitudes (lb has it) moves every probability by as much, twice in the quotient.
    move = 2 * lb[..., None]
    po.check("out", out, o, ob + move * (p @ _wide(v, 2).abs()))
    po.check("lse", lse, l, lb)
    (wq, bq), (wk, bk), (wv, bv) = po.attention_bwd(q.double(), _wide(k, 2), _wide(v, 2), do.double(), see, None,
                                                    ob + move * (p @ _wide(v, 2).abs()))
    scale = d ** -0.5
    spread = p * ((do.double() @ _wide(v, 2).mT).abs() + (do.double() * o).sum(-1, keepdim=True).abs()) * move
    fold = lambda x: x.view(1, 1, 2, n, d).sum(2)  # noqa: E731
    po.check("dq", dq, wq, bq + scale * spread @ _wide(k, 2).abs())
    po.check("dk", dk, fold(wk), fold(bk + scale * spread.mT @ q.double().abs()))
    po.check("dv", dv, fold(wv), fold(bv + (p * move).mT @ do.double().abs()))


def test_offsets_beyond_32_bits():
    """A million positions of 32 heads of 128: 2^32 elements of q and out; the last rows of the
    last head, and the first's."""
    moba = _moba()
    n, d, window, sink = 1 << 20, 128, 128, 3
    g = torch.Generator("cuda").manual_seed(31)
    q = torch.empty(1, 32, n, d, dtype=torch.bfloat16, device="cuda")
    for h in range(32):
        q[0, h].copy_(torch.randn(n, d, generator=g, device="cuda"))
    k, v = (torch.randn(1, 2, n, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    out, lse = moba.swa_attn_fwd(q, k, v, window, sink=sink)
    cos, sin = torch.ones(n, 8, device="cuda"), torch.zeros(n, 8, device="cuda")
    same, _ = moba.qk_norm_rope_fwd(q, k, cos, sin)
    assert moba.device_status() == 0
    assert torch.equal(same[0, 31, -300:], q[0, 31, -300:]) and torch.equal(same[0, 0, :9], q[0, 0, :9])
    at = torch.cat([torch.arange(sink, device="cuda"), torch.arange(n - 400, n, device="cuda")])
    see = torch.cat([torch.ones(200, sink, dtype=torch.bool, device="cuda"),
                     po.visible(200, 400, window, 0, "cuda")], 1)
    for h in (0, 15, 31):
        kk, vv = k[0, h // 16, at].double(), v[0, h // 16, at].double()
        o, l, _, ob, lb = po.attention(q[0, h, -200:].double(), kk, vv, see)
        po.check("out", out[0, h, -200:], o, ob)
        po.check("lse", lse[0, h, -200:], l, lb)


def test_backward_with_a_scale_repeats_bit_for_bit():
    moba = _moba()
    (q, k, v, do, out, lse), grads = _bwd(1, 4, 2, 1500, 64, 90, 7, scale=0.3)
    for _ in range(3):
        again = moba.swa_attn_bwd(q, k, v, out, lse, do, 90, 7, 0.3)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_backward_equals_differences_of_the_forward():
    """sum(dO out) along a direction, from the kernel's own forward in steps large enough to
    stand above its bf16 rounding: out is off by at most 2^-8 of itself and of p |v| (a sum
    of 2 n d such errors with random signs), the step is 1/4, so the quotient is good to a few
    per cent of the gradient's norm along it."""
    moba = _moba()
    q, k, v, do = _inputs(1, 2, 1, 200, 200, 64, 5)
    out, lse = moba.swa_attn_fwd(q, k, v, 50, sink=3)
    dq, dk, dv = moba.swa_attn_bwd(q, k, v, out, lse, do, 50, sink=3)

    def loss(v2):
        o, _ = moba.swa_attn_fwd(q, k, v2, 50, sink=3)
        return float((o.double() * do.double()).sum())

    u = torch.randn(v.shape, generator=torch.Generator("cuda").manual_seed(6), device="cuda").bfloat16()
    up, down = (v + 0.25 * u).bfloat16(), (v - 0.25 * u).bfloat16()
    got, want = loss(up) - loss(down), float((dv.double() * (up.double() - down.double())).sum())
    # (The loss is linear in v: no curvature.)  Each of the outputs, 2 x 200 x 64 of
    # magnitude below 1 against dO of 1, carries up to 2^-7; the sum of their errors, of
    # random sign, stays within six deviations of 2^-7 sqrt(2 x 25600).
    assert abs(got - want) <= 6 * 2.0 ** -7 * (2 * 25600) ** 0.5, (got, want)


def test_on_another_stream_and_in_a_graph():
    moba = _moba()
    q, k, v, do = _inputs(1, 4, 2, 700, 700, 80, 8)
    out, lse = moba.swa_attn_fwd(q, k, v, 100, sink=5)
    want = moba.swa_attn_bwd(q, k, v, out, lse, do, 100, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = moba.swa_attn_fwd(q, k, v, 100, sink=5, stream=side)
    got = moba.swa_attn_bwd(q, k, v, o2, l2, do, 100, 5, stream=side)
    side.synchronize()
    assert torch.equal(out, o2) and all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, l3 = moba.swa_attn_fwd(q, k, v, 100, sink=5)
        got = moba.swa_attn_bwd(q, k, v, o3, l3, do, 100, 5)
    for _ in range(2):
        for t in (o3, l3, *got):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o3) and all(torch.equal(a, b) for a, b in zip(want, got))
    assert moba.device_status() == 0


def test_results_of_another_stream_stay_until_they_are_read():
    """A result allocated on the call's stream is read on the caller's behind a long kernel
    and dropped before that: its memory must not be handed out again meanwhile."""
    moba = _moba()
    q, k, v, _ = _inputs(1, 8, 8, 2000, 2000, 128, 9)
    want, _ = moba.swa_attn_fwd(q, k, v, 100, sink=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = moba.swa_attn_fwd(q, k, v, 100, sink=5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(50_000_000)
    got = torch.empty_like(out)
    got.copy_(out)
    del out
    with torch.cuda.stream(side):
        junk = [torch.full_like(q, 9.0) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(junk) == 4


def test_forward_without_the_compiled_binding(monkeypatch):
    """Another torch finds no binding; the forward then goes through ctypes, like the prefill."""
    moba = _moba()
    q, k, v, _ = _inputs(2, 4, 2, 300, 500, 80, 9)
    want = [moba.swa_attn_fwd_chunk(q, k, v, 77, 0.2, sink=s) for s in (0, 5)]

    class Missing:
        def __getattr__(self, name):
            raise ImportError(name)

    monkeypatch.setattr(moba, "_binding", Missing())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s, (out, lse) in zip((0, 5), want):
        for stream in (None, side):
            o, l = moba.swa_attn_fwd_chunk(q, k, v, 77, 0.2, stream=stream, sink=s)
            torch.cuda.synchronize()
            assert torch.equal(o, out) and torch.equal(l, lse)
    with pytest.raises(ValueError, match="k has shape"):
        moba.swa_attn_fwd(q, k[:1], v, 77)
    with pytest.raises(ImportError):
        moba.swa_attn_bwd(q, q, q, q, lse, q, 77)


@pytest.mark.parametrize("d,hq,hkv,n,nk,window", [(64, 2, 1, 900, 900, 200), (80, 2, 2, 333, 900, 128),
                                                  (128, 4, 2, 900, 900, 200), (128, 2, 1, 700, 700, 5000)])
def test_forward_of_the_band_alone(d, hq, hkv, n, nk, window):
    """No sinks: the float64 band."""
    _fwd(1, hq, hkv, n, nk, d, window, 0, seed=window)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("hq,hkv,n,window,sink", [(2, 2, 1000, 1000, 0), (4, 2, 1100, 500, 4), (8, 2, 900, 130, 140),
                                                  (2, 1, 700, 5, 1)])
def test_whole_gradients(d, hq, hkv, n, window, sink):
    """Each gradient as a whole: the bounds of single values add up magnitudes, which at wide
    windows leaves room for errors of D or of the sums that the 2-norm does not."""
    moba = _moba()
    q, k, v, do = _inputs(2, hq, hkv, n, n, d, n + d)
    out, lse = moba.swa_attn_fwd(q, k, v, window, sink=sink)
    got = moba.swa_attn_bwd(q, k, v, out, lse, do, window, sink)
    assert moba.device_status() == 0
    G, see = hq // hkv, po.visible(n, n, window, sink, "cuda")
    args = q.double(), _wide(k, G), _wide(v, G), do.double(), see
    (wq, _), (wk, _), (wv, _) = po.attention_bwd(*args)
    want = wq, wk.view(2, hkv, G, n, d).sum(2), wv.view(2, hkv, G, n, d).sum(2)
    bounds = list(po.attention_bwd_norms(*args))
    if G > 1:   # (stored once, after the sum over the heads: its rounding is of the sum)
        bounds[1:] = [(b ** 2 + (po.BF16 * float(w.norm())) ** 2) ** 0.5 for b, w in zip(bounds[1:], want[1:])]
    for name, x, w, b in zip(("dq", "dk", "dv"), got, want, bounds):
        err = float((x.double() - w).norm())
        assert err <= b, (name, err, b, float(w.norm()))


@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("d", [64, 80, 128])
def test_gradients_equal_differences_of_the_forward(name, d):
    """sum(dO out) of the kernel's own forward, in a step along the kernel's gradient, where the
    loss changes most: by many times what its roundings leave open."""
    moba = _moba()
    hq, hkv, n, window, sink = 2, 1, 300, 50, 3
    x = dict(zip(("q", "k", "v", "do"), _inputs(1, hq, hkv, n, n, d, 5)))
    do, see, scale = x["do"].double(), po.visible(n, n, window, sink, "cuda"), d ** -0.5
    out, lse = moba.swa_attn_fwd(x["q"], x["k"], x["v"], window, sink=sink)
    grads = dict(zip(("q", "k", "v"), moba.swa_attn_bwd(x["q"], x["k"], x["v"], out, lse, x["do"], window, sink)))

    def plain(y):
        """The loss in float64, and how far the kernel's may be from it: the stored out, P before
        its product, and float32 scores and sums (2^-13 of the terms)."""
        q, k, v = y["q"].double(), _wide(y["k"], hq // hkv), _wide(y["v"], hq // hkv)
        o, _, p, _, _ = po.attention(q, k, v, see)
        terms = (p * (do @ v.mT).abs()).sum()
        return float((do * o).sum()), float(po.BF16 * ((do * o).abs().sum() + terms) + 2.0 ** -13 * terms)

    def loss(y):
        return float((moba.swa_attn_fwd(y["q"], y["k"], y["v"], window, sink=sink)[0].double() * do).sum())

    g = grads[name].double()
    step = dict(q=0.5, k=0.5, v=2.0)[name]
    up, down = (dict(x, **{name: (x[name].double() + s * step * g).bfloat16()}) for s in (1, -1))
    way = up[name].double() - down[name].double()
    want = float((g * way).sum())
    (lu, eu), (ld, ed) = plain(up), plain(down)
    # The loss bends along q and k: the formula's difference misses its own gradient by as much.
    args = x["q"].double(), _wide(x["k"], hq // hkv), _wide(x["v"], hq // hkv), do, see
    exact = dict(zip("qkv", (w for w, _ in po.attention_bwd(*args))))[name]
    if name != "q":
        exact = exact.view(1, hkv, hq // hkv, n, d).sum(2)
    want += lu - ld - float((exact * way).sum())
    # The gradient itself: its whole error (twice the heads' norms) along the way.
    norm = 2 * dict(zip("qkv", po.attention_bwd_norms(*args)))[name] * float(way.norm())
    tol = eu + ed + norm
    assert tol < 0.1 * want, (tol, want)
    assert abs(loss(up) - loss(down) - want) <= tol, (loss(up) - loss(down), want, tol)


def test_backward_offsets_beyond_32_bits():
    """The same sizes in the backward: the last rows and keys of the last heads, and the sinks'
    keys, which every row of their sixteen heads sees."""
    moba = _moba()
    n, d, window, sink, hq, hkv = 1 << 20, 128, 128, 3, 32, 2
    G, scale, m = hq // hkv, d ** -0.5, 400
    g = torch.Generator("cuda").manual_seed(33)

    def rand(heads):
        x = torch.empty(1, heads, n, d, dtype=torch.bfloat16, device="cuda")
        for h in range(heads):
            x[0, h].copy_(torch.randn(n, d, generator=g, device="cuda"))
        return x

    q, do, k, v = rand(hq), rand(hq), rand(hkv), rand(hkv)
    out, lse = moba.swa_attn_fwd(q, k, v, window, sink=sink)
    dq, dk, dv = moba.swa_attn_bwd(q, k, v, out, lse, do, window, sink)
    assert moba.device_status() == 0
    # The last m - window rows of the last KV head's query heads against the keys that they see.
    at = torch.cat([torch.arange(sink, device="cuda"), torch.arange(n - m, n, device="cuda")])
    see = torch.cat([torch.ones(m, sink, dtype=torch.bool, device="cuda"), po.visible(m, m, window, 0, "cuda")], 1)
    keep = m - window
    kk, vv = (x[0, -1, at].double().expand(G, -1, -1) for x in (k, v))
    args = q[0, -G:, -m:].double(), kk, vv, do[0, -G:, -m:].double(), see
    o, _, _, ob, _ = po.attention(*args[:3], see)
    (wq, bq), (wk, bk), (wv, bv) = po.attention_bwd(*args, None, ob)
    po.check("dq", dq[0, -G:, -keep:], wq[:, -keep:], bq[:, -keep:])
    # (Keys of the last window - 1 positions are seen by these rows alone, and by all of them.)
    last = window - 1
    po.check("dk", dk[0, -1, -last:], wk.sum(0)[-last:], bk.sum(0)[-last:])
    po.check("dv", dv[0, -1, -last:], wv.sum(0)[-last:], bv.sum(0)[-last:])
    for hk in (0, hkv - 1):
        ks, vs = k[0, hk, :sink].double(), v[0, hk, :sink].double()
        want, bound = ([torch.zeros(sink, d, dtype=torch.float64, device="cuda") for _ in range(2)] for _ in range(2))
        for h in range(hk * G, (hk + 1) * G):
            for a in range(0, n, n // 4):
                rows = slice(a, a + n // 4)
                qq, oo, gg = q[0, h, rows].double(), out[0, h, rows].double(), do[0, h, rows].double()
                i = torch.arange(a, a + n // 4, device="cuda")
                p = torch.exp(scale * qq @ ks.T - lse[0, h, rows].double()[:, None])
                p = torch.where(i[:, None] >= torch.arange(sink, device="cuda"), p, 0.0)
                dz = p * (gg @ vs.T - (gg * oo).sum(-1, keepdim=True))
                for x, y, w in ((want[0], bound[0], (dz, qq, scale)), (want[1], bound[1], (p, gg, 1.0))):
                    x += w[2] * w[0].T @ w[1]
                    # (Every dz and P is rounded, and the squares of the errors add up; D is the one
                    # that the kernel takes, float32 statistics and sums err by far less.)
                    y += (w[2] * po.BF16) ** 2 * w[0].square().T @ w[1].square()
        for name, x, w, b in (("dk", dk, want[0], bound[0]), ("dv", dv, want[1], bound[1])):
            err = x[0, hk, :sink].double() - w
            assert float(err.norm()) <= float((b.sum() + (po.BF16 * w).square().sum()).sqrt()), (name, hk)
