"""The paged cache: appending to it and attending one token over it, against the float64
formulas, value by value (tests/plain_ops.py derives the bounds); and the operators in a
row, as a server and as a training step use them."""
import math

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


class Cache:
    """Scattered pages of sequences of the given lengths, filled with random values; the
    slots that no sequence owns hold NaN."""

    def __init__(self, lens, hkv, page, d, seed=0, layout="hnd", spare=2, width=None):
        g = torch.Generator("cuda").manual_seed(seed)
        need = [-(-n // page) for n in lens]
        total = sum(need) + spare
        shape = (total, hkv, page, d) if layout == "hnd" else (total, page, hkv, d)
        view = (lambda x: x) if layout == "hnd" else (lambda x: x.permute(0, 2, 1, 3))
        self.k, self.v = (view(torch.randn(shape, generator=g, device="cuda").bfloat16()) for _ in range(2))
        perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed))
        width = width or max(1, max(need))
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for s, m in enumerate(need):
            self.table[s, :m] = perm[at:at + m].int()
            at += m
        owned = torch.zeros(total, page, dtype=torch.bool)
        for s, n in enumerate(lens):
            for j in range(n):
                owned[self.table[s, j // page], j % page] = True
        self.owned = owned.cuda()
        for x in (self.k, self.v):
            x.copy_(torch.where(self.owned[:, None, :, None], x.float(), math.nan).bfloat16())
        self.table = self.table.cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")


def _decode(lens, hq, hkv, page, d, window=0, sink=0, seed=0, layout="hnd", scale=0.0, width=None, qscale=1.0):
    moba = _moba()
    c = Cache(lens, hkv, page, d, seed, layout, width=width)
    q = (qscale * torch.randn(len(lens), hq, d, generator=torch.Generator("cuda").manual_seed(seed + 1),
                              device="cuda")).bfloat16()
    out, lse = moba.paged_decode_attn(q, c.k, c.v, c.table, c.lens, window, sink, scale)
    assert moba.device_status() == 0
    G = hq // hkv
    for s, n in enumerate(lens):
        if n == 0:
            assert not out[s].any() and torch.isneginf(lse[s]).all()
            continue
        k, v = (po.gather_pages(x, c.table[s], n).repeat_interleave(G, 0) for x in (c.k, c.v))
        o, l, _, ob, lb = po.attention(q[s].double()[:, None], k, v, po.visible(1, n, window, sink, "cuda"),
                                       scale or None)
        po.check(f"out {s}", out[s], o[:, 0], ob[:, 0])
        po.check(f"lse {s}", lse[s], l[:, 0], lb[:, 0])
    return c, q, out, lse


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [0, 3, 0, 250, 1, 64], [3001]])
@pytest.mark.parametrize("page,layout", [(16, "hnd"), (24, "nhd"), (1, "nhd")])
def test_decode(d, lens, page, layout):
    _decode(lens, 4, 2, page, d, seed=len(lens), layout=layout)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (8, 1), (16, 1), (17, 1), (40, 1), (32, 8), (5, 5)])
def test_decode_of_every_group_size(hq, hkv):
    _decode([700, 33, 129], hq, hkv, 32, 128, seed=hq)


@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (100, 0), (100, 4), (64, 130), (5000, 4), (333, 16)])
def test_decode_with_a_window_and_sinks(window, sink):
    _decode([1, 64, 101, 400, 1999], 6, 3, 48, 80, window, sink, seed=window)


def test_decode_of_many_and_uneven_sequences():
    r = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 300, (200,), generator=r).tolist()
    lens[17], lens[150] = 20000, 0
    _decode(lens, 8, 2, 16, 64, seed=3, layout="nhd", width=2000)
    _decode([0] * 5, 8, 2, 16, 64)


def test_decode_with_a_scale_and_large_scores():
    """Scores of hundreds: one key takes all of the weight, and the running maximum rises
    again and again."""
    _decode([900, 31], 4, 1, 32, 128, scale=1.5, qscale=4.0, seed=2)


def test_decode_leaves_out_bad_pages_and_lengths():
    moba = _moba()
    c, q, out, lse = _decode([200, 70, 90], 4, 2, 16, 64, seed=5)
    table = c.table.clone()
    table[0, 3], table[0, 7] = c.k.shape[0], -1
    got, _ = moba.paged_decode_attn(q, c.k, c.v, table, c.lens)
    assert moba.device_status() == -10 and moba.device_status() == 0
    assert torch.equal(got[1:], out[1:])
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[48:64] = False
    keep[112:128] = False
    k, v = (po.gather_pages(x, c.table[0], 200).repeat_interleave(2, 0) for x in (c.k, c.v))
    o, _, _, ob, _ = po.attention(q[0].double()[:, None], k, v, keep[None])
    po.check("out", got[0], o[:, 0], ob[:, 0])
    lens = c.lens.clone()
    lens[1] = -5
    got, gl = moba.paged_decode_attn(q, c.k, c.v, c.table, lens)
    assert moba.device_status() == -10
    assert not got[1].any() and torch.isneginf(gl[1]).all()
    # (The tiles are dealt out anew: the same sums in another order.)
    k, v = (po.gather_pages(x, c.table[2], 90).repeat_interleave(2, 0) for x in (c.k, c.v))
    o, _, _, ob, _ = po.attention(q[2].double()[:, None], k, v, torch.ones(1, 90, dtype=torch.bool, device="cuda"))
    po.check("out", got[2], o[:, 0], ob[:, 0])
    # Longer than the table: the table's end is the length.
    whole = torch.tensor([13 * 16], dtype=torch.int32, device="cuda")
    full = Cache([13 * 16], 2, 16, 64, 1)
    a, _ = moba.paged_decode_attn(q[:1], full.k, full.v, full.table, whole)
    b, _ = moba.paged_decode_attn(q[:1], full.k, full.v, full.table, whole + 1000)
    assert moba.device_status() == -10 and torch.equal(a, b)


def test_decode_of_strided_queries_into_strided_outputs():
    moba = _moba()
    c, q, out, lse = _decode([130, 260], 4, 2, 16, 128, seed=6)
    wide = torch.zeros(2, 9, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:7] = q
    dst = torch.full((2, 6, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    moba.paged_decode_attn(wide[:, 3:7], c.k, c.v, c.table, c.lens, out=dst[:, 1:5])
    assert torch.equal(dst[:, 1:5], out) and (dst[:, 0] == 5).all() and (dst[:, 5] == 5).all()


def test_two_graphs_share_a_workspace():
    """Graphs captured over one workspace and replayed in turn on one stream, lengths that
    change between replays: nothing is carried from call to call."""
    moba = _moba()
    a = Cache([500, 40], 2, 16, 64, 1)
    b = Cache([9, 1000, 77], 2, 16, 64, 2)
    qa = torch.randn(2, 8, 64, device="cuda").bfloat16()
    qb = torch.randn(3, 8, 64, device="cuda").bfloat16()
    ws = torch.empty(moba.paged_decode_workspace_size(3, 8, 2, 64), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    run = lambda q, c, w=None: moba.paged_decode_attn(q, c.k, c.v, c.table, c.lens, workspace=w)  # noqa: E731
    graphs = []
    for q, c in ((qa, a), (qb, b)):
        run(q, c, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run(q, c, ws)
        graphs.append((g, got, q, c))
    for turn in range(3):
        for g, got, q, c in graphs:
            g.replay()
            want = run(q, c)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            c.lens -= 3
    assert moba.device_status() == 0


def test_pages_beyond_32_bits():
    """A cache of 2.3 x 10^9 elements: pages at its end, appended to and attended."""
    moba = _moba()
    pages, hkv, page, d, n = 140000, 8, 16, 128, 100
    kp = torch.empty(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    vp = torch.empty(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    table = (pages - 1 - torch.arange(7, dtype=torch.int32, device="cuda") * 1111)[None].contiguous()
    table[0, 3] = 0
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(41)
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").bfloat16() for h in (16, hkv, hkv))
    moba.kv_append(k, v, kp, vp, table, lens, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    assert torch.equal(po.gather_pages(kp, table[0], n), k.double().transpose(0, 1))
    assert torch.equal(po.gather_pages(vp, table[0], n), v.double().transpose(0, 1))
    out, lse = moba.paged_decode_attn(q[-1:], kp, vp, table, lens)
    assert moba.device_status() == 0
    kk, vv = (x.double().transpose(0, 1).repeat_interleave(2, 0) for x in (k, v))
    o, l, _, ob, lb = po.attention(q[-1].double()[:, None], kk, vv, torch.ones(1, n, dtype=torch.bool, device="cuda"))
    po.check("out", out[0], o[:, 0], ob[:, 0])
    po.check("lse", lse[0], l[:, 0], lb[:, 0])


def test_shared_pages():
    """Sequences that share a prefix's pages, and a page named twice in one sequence."""
    moba = _moba()
    c, q, out, lse = _decode([64, 64], 4, 2, 16, 64, seed=8)
    table = c.table.clone()
    table[1, :3] = table[0, :3]
    table[1, 3] = table[1, 0]
    got, gl = moba.paged_decode_attn(q, c.k, c.v, table, c.lens)
    assert moba.device_status() == 0 and torch.equal(got[0], out[0])
    k, v = (po.gather_pages(x, table[1], 64).repeat_interleave(2, 0) for x in (c.k, c.v))
    o, _, _, ob, _ = po.attention(q[1].double()[:, None], k, v, torch.ones(1, 64, dtype=torch.bool, device="cuda"))
    po.check("out", got[1], o[:, 0], ob[:, 0])


def test_the_binding_names_what_is_wrong():
    moba = _moba()
    c = Cache([20, 3], 2, 16, 64)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    for match, call in (
            ("q must be torch.bfloat16", lambda: moba.paged_decode_attn(q.float(), c.k, c.v, c.table, c.lens)),
            ("seq_lens must be torch.int32", lambda: moba.paged_decode_attn(q, c.k, c.v, c.table, c.lens.long())),
            ("page_table has shape", lambda: moba.paged_decode_attn(q[:1], c.k, c.v, c.table, c.lens[:1])),
            ("v_pages has shape", lambda: moba.paged_decode_attn(q, c.k, c.v[:1], c.table, c.lens)),
            ("k_pages has shape", lambda: moba.paged_decode_attn(q[..., :32], c.k, c.v, c.table, c.lens)),
            ("page_table must be contiguous", lambda: moba.paged_decode_attn(q, c.k, c.v, c.table.repeat(1, 2)[:, ::2],
                                                                             c.lens)),
            ("head dimension", lambda: moba.paged_decode_attn(q.repeat(1, 1, 2)[..., ::2], c.k, c.v, c.table, c.lens)),
            ("lse must be a CUDA tensor", lambda: moba.paged_decode_attn(q, c.k, c.v, c.table, c.lens,
                                                                         lse=torch.zeros(2, 4))),
            ("cos and sin", lambda: moba.kv_append(q[:, :2], q[:, :2], c.k, c.v, c.table, c.lens, cos=torch.zeros(9, 8, device="cuda"))),
            ("need q", lambda: moba.kv_append(q[:, :2], q[:, :2], c.k, c.v, c.table, c.lens, q_out=q))):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(moba.MobaError) as e:
        moba.paged_decode_attn(q, c.k, c.v, c.table, c.lens, window=-2)
    assert e.value.code == -4
    torch.cuda.synchronize()


# ------------------------------------------------------------------ append

def _append(news, lens, hq, hkv, page, d, rot, norm, inter, layout="hnd", pad=0, seed=0, cu_null=False):
    moba = _moba()
    c = Cache(lens, hkv, page, d, seed, layout)
    c.k.fill_(9)
    c.v.fill_(9)
    g = torch.Generator("cuda").manual_seed(seed + 1)
    T = sum(news)
    x = torch.randn(T + pad, hq + 2 * hkv, d, generator=g, device="cuda").bfloat16()
    q, k, v = x.split([hq, hkv, hkv], 1)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2)) if norm else (None, None)
    cos, sin = _table(max(lens) + 1, rot) if rot else (None, None)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    qo = torch.full((T + pad, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    cut = None if cu_null else torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = moba.kv_append(k, v, c.k, c.v, c.table, c.lens, cut, cos, sin, wk, EPS, inter, q, wq, qo)
    assert got is qo and moba.device_status() == 0
    at = [(s, lens[s] - n + r) for s, n in enumerate(news) for r in range(n)]
    touched = torch.zeros(c.k.shape[0], page, dtype=torch.bool)
    table = c.table.cpu()
    if at:
        pos = torch.tensor([p for _, p in at], device="cuda")
        if rot:
            cc, ss = cos.double()[pos][:, None], sin.double()[pos][:, None]
        else:
            cc = ss = torch.zeros(T, 1, 0, dtype=torch.float64, device="cuda")
        for name, src, wt, dst in (("q", q, wq, qo[:T]), ("k", k, wk, None)):
            want, bound = po.norm_rope(src[:T].double(), None if wt is None else wt.double(), cc, ss, inter, EPS)
            if dst is None:
                dst = torch.stack([c.k[table[s, p // page], :, p % page] for s, p in at])
            po.check(name, dst, want, bound)
        assert torch.equal(torch.stack([c.v[table[s, p // page], :, p % page] for s, p in at]), v[:T])
        for s, p in at:
            touched[table[s, p // page], p % page] = True
    # Nothing else is touched: other slots, and the queries behind the last sequence.
    rest = ~touched.cuda()[:, None, :, None].expand(c.k.shape)
    assert (c.k[rest] == 9).all() and (c.v[rest] == 9).all() and (qo[T:] == 9).all()


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("news,lens,pad", [([1], [1], 0), ([0, 5, 0, 0, 40, 1], [0, 5, 7, 0, 100, 33], 3),
                                           ([200], [777], 130), ([2] * 70, list(range(2, 72)), 5)])
@pytest.mark.parametrize("page,layout", [(16, "hnd"), (24, "nhd"), (1, "hnd")])
def test_append(d, news, lens, pad, page, layout):
    inter = d == 80
    _append(news, lens, 6, 3, page, d, 32 if page == 24 else d, page != 1, inter, layout, pad, seed=d)


def test_append_one_token_each_without_offsets():
    lens = [5, 1, 64, 65, 200]
    _append([1] * 5, lens, 32, 8, 16, 128, 128, True, False, cu_null=True)
    _append([1] * 5, lens, 1, 1, 16, 64, 0, False, False, cu_null=True)
    _append([1] * 5, lens, 1, 1, 16, 64, 0, True, True, cu_null=True)


def test_append_of_nothing():
    moba = _moba()
    c = Cache([20], 2, 16, 64)
    x = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert moba.kv_append(x, x, c.k, c.v, c.table, c.lens, cu) is None
    assert moba.device_status() == 0


def test_append_leaves_out_what_has_no_place():
    """A page that is not there, a position before the first, one behind the table, one
    without angles, and tokens before the first offset: nothing is written for them."""
    moba = _moba()
    page, d = 16, 64
    c = Cache([40, 20, 30, 10], 1, page, d, 4)
    c.k.fill_(9)
    c.v.fill_(9)
    cos, sin = _table(39, d)
    cu = torch.tensor([2, 6, 8, 10, 12], dtype=torch.int32, device="cuda")
    lens = torch.tensor([40, 20, 1, 1000], dtype=torch.int32, device="cuda")
    table = c.table.clone()
    table[1, 1] = 1 << 30
    x = torch.randn(15, 1, d, device="cuda").bfloat16()
    moba.kv_append(x, x, c.k, c.v, table, lens, cu, cos, sin)
    assert moba.device_status() == -10
    # Sequence 0: positions 36 .. 39, the last without angles.  1: positions 18, 19 on the bad
    # page.  2: positions -1 and 0.  3: positions 998, 999 behind the table.
    t = c.table.cpu()
    ok = {2: (0, 36), 3: (0, 37), 4: (0, 38), 9: (2, 0)}
    touched = torch.zeros(c.v.shape[0], page, dtype=torch.bool, device="cuda")
    for tok, (s, p) in ok.items():
        assert torch.equal(c.v[t[s, p // page], :, p % page], x[tok])
        touched[t[s, p // page], p % page] = True
    assert (c.v[~touched[:, None, :, None].expand(c.v.shape)] == 9).all()
    assert (c.k[~touched[:, None, :, None].expand(c.k.shape)] == 9).all()


@pytest.mark.parametrize("which", ["page", "page id below 0", "behind the table", "angles", "position"])
def test_append_writes_no_query_of_a_token_without_a_place(which):
    """The token's key, value and query row are left as they were; its neighbours' are written."""
    moba = _moba()
    page, d, hq = 16, 80, 3
    c = Cache([40, 20, 30], 1, page, d, 14)
    for x in (c.k, c.v):
        x.fill_(9)
    cos, sin = _table(1 << 10, d)
    table, lens = c.table.clone(), torch.tensor([40, 20, 30], dtype=torch.int32, device="cuda")
    if which == "page":
        table[1, 1] = c.k.shape[0]
    elif which == "page id below 0":
        table[1, 1] = -1
    elif which == "behind the table":
        lens[1] = table.shape[1] * page + 1
    elif which == "angles":
        lens[1] = (1 << 10) + 1
    else:
        lens[1] = 0
    x = torch.randn(3, hq + 2, d, generator=torch.Generator("cuda").manual_seed(15), device="cuda").bfloat16()
    q, k, v = x.split([hq, 1, 1], 1)
    qo = torch.full((3, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    moba.kv_append(k, v, c.k, c.v, table, lens, None, cos, sin, q=q, q_out=qo)
    assert moba.device_status() == -10
    pos = torch.tensor([39, 29], device="cuda")
    want, bound = po.norm_rope(q[[0, 2]].double(), None, cos.double()[pos][:, None], sin.double()[pos][:, None], False, EPS)
    po.check("q", qo[[0, 2]], want, bound)
    assert (qo[1] == 9).all()
    written = (c.v != 9).any(1).any(-1).nonzero().tolist()
    assert sorted(written) == sorted([[int(table[s, p // page]), p % page] for s, p in ((0, 39), (2, 29))])


# ------------------------------------------------------------------ in a row

@pytest.mark.parametrize("window,sink", [(0, 0), (50, 4)])
def test_a_server_prefills_and_decodes(window, sink):
    """A prompt goes through the cache in chunks and its last tokens one by one; each decoded
    row is the row of one prefill over the same rotated keys."""
    moba = _moba()
    hq, hkv, d, n, page, steps = 8, 2, 128, 150, 16, 4
    g = torch.Generator("cuda").manual_seed(11)
    x = torch.randn(2, n, hq + 2 * hkv, d, generator=g, device="cuda").bfloat16()
    w = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16()
    cos, sin = _table(n, d)
    q, k, v = (t.permute(0, 2, 1, 3) for t in x.split([hq, hkv, hkv], 2))
    qr, kr = moba.qk_norm_rope_fwd(q, k, cos, sin, None, w, w, EPS)
    want, lse = moba.swa_attn_fwd(qr, kr, v, window or n, sink=sink)
    c = Cache([n, n], hkv, page, d, 12)
    ws = torch.empty(moba.paged_decode_workspace_size(2, hq, hkv, d), dtype=torch.uint8, device="cuda")
    done = 0
    for chunk in (70, n - steps - 70):
        part = x[:, done:done + chunk].reshape(2 * chunk, hq + 2 * hkv, d)
        done += chunk
        pq, pk, pv = part.split([hq, hkv, hkv], 1)
        lens = torch.full((2,), done, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, chunk, 2 * chunk], dtype=torch.int32, device="cuda")
        moba.kv_append(pk, pv, c.k, c.v, c.table, lens, cu, cos, sin, w, EPS)
    for t in range(n - steps, n):
        pq, pk, pv = x[:, t].split([hq, hkv, hkv], 1)
        lens = torch.full((2,), t + 1, dtype=torch.int32, device="cuda")
        qt = moba.kv_append(pk, pv, c.k, c.v, c.table, lens, None, cos, sin, w, EPS, q=pq, q_weight=w)
        assert torch.equal(qt, qr[:, :, t])
        out, l = moba.paged_decode_attn(qt, c.k, c.v, c.table, lens, window, sink, workspace=ws)
        for s in range(2):
            kk, vv = (y[s, :, :t + 1].double().repeat_interleave(hq // hkv, 0) for y in (kr, v))
            o, ll, _, ob, lb = po.attention(qt[s].double()[:, None], kk, vv, po.visible(1, t + 1, window, sink, "cuda"))
            po.check("decode", out[s], o[:, 0], ob[:, 0])
            po.check("prefill", want[s, :, t], o[:, 0], ob[:, 0])
            po.check("lse", l[s], ll[:, 0], lb[:, 0])
            po.check("lse", lse[s, :, t], ll[:, 0], lb[:, 0])
    assert moba.device_status() == 0


def test_a_training_step_through_norm_rotation_and_attention():
    """Gradients of sum(dO out) through the attention and the norm to the projections' results
    and the norm weights, against automatic differentiation in float64.  Between the two
    steps q, k, their gradients, P and dz are rounded to bf16 (2^-8 each, random signs):
    the whole gradients are within 1% in the 2-norm."""
    moba = _moba()
    hq, hkv, d, n, window, sink = 4, 2, 80, 300, 64, 3
    g = torch.Generator("cuda").manual_seed(13)
    q, k, v, do = (torch.randn(1, h, n, d, generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv, hq))
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    cos, sin = _table(n, 32)
    qr, kr = moba.qk_norm_rope_fwd(q, k, cos, sin, None, w, w, EPS)
    out, lse = moba.swa_attn_fwd(qr, kr, v, window, sink=sink)
    dqr, dkr, dv = moba.swa_attn_bwd(qr, kr, v, out, lse, do, window, sink)
    dq, dk, dwq, dwk = moba.qk_norm_rope_bwd(dqr, dkr, q, k, cos, sin, None, w, w, EPS)
    assert moba.device_status() == 0
    lq, lk, lv = (t.double().requires_grad_() for t in (q, k, v))
    lwq, lwk = (w.double().requires_grad_() for _ in range(2))
    c, s = cos.double(), sin.double()
    a = po.norm_rope(lq, lwq, c, s, False, EPS)[0]
    b = po.norm_rope(lk, lwk, c, s, False, EPS)[0].repeat_interleave(2, 1)
    z = (a @ b.mT * d ** -0.5).masked_fill(~po.visible(n, n, window, sink, "cuda"), -math.inf)
    loss = (torch.softmax(z, -1) @ lv.repeat_interleave(2, 1) * do.double()).sum()
    want = torch.autograd.grad(loss, (lq, lk, lv, lwq, lwk))
    for name, x, y in zip(("dq", "dk", "dv", "dwq", "dwk"), (dq, dk, dv, dwq, dwk), want):
        rel = float((x.double() - y).norm() / y.norm())
        assert rel <= 1e-2, (name, rel)
