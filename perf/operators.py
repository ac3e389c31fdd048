"""What is measured of the serving and training operators around the attention kernels.

Four operators, one state and one pass each:

  swa     sliding-window attention whose first ``sink`` tokens stay visible, forward
          (``train`` 0) or forward and backward (``train`` 1)
  decode  attention of one new token per sequence over a paged key-value cache
  append  new tokens' keys and values into a paged cache, keys (and queries) normalised
          per head and rotated to their positions on the way
  qknr    norms of queries and keys per head with the position rotation, forward
          (``bwd`` 0) or backward (``bwd`` 1)

Where ``own`` is false, ``run`` computes them from elementary torch operations in 32 bits;
where it is true it makes the calls of this package.
"""
import math
import random

import torch

own = False

_EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One short prompt of a small sliding-window layer: a launch, latency counts.
        dict(name="swa_prompt_1000", op="swa", train=0, batch=1, hq=4, hkv=2, n=1000, nk=1000, d=64,
             window=200, sink=4),
        # A whole prefill of the 16K sliding-window workload (32 heads of 80, window 4096)
        # whose first four tokens stay visible.
        dict(name="swa_prefill_16k", op="swa", train=0, batch=1, hq=32, hkv=32, n=16384, nk=16384, d=80,
             window=4096, sink=4),
        # A training step through a GQA layer with the hybrid workload's heads and window
        # (8 query and 4 KV heads of 128, window 512) at an odd length, sinks past one tile.
        dict(name="swa_train_gqa_8k", op="swa", train=1, batch=2, hq=8, hkv=4, n=8191, nk=8191, d=128,
             window=512, sink=130),
        # A training step through the 16K sliding-window layer.
        dict(name="swa_train_16k", op="swa", train=1, batch=1, hq=32, hkv=32, n=16384, nk=16384, d=80,
             window=4096, sink=4),
        # One chat continuing at 4K tokens: latency of a single decode step.
        dict(name="decode_one_4k", op="decode", batch=1, hq=32, hkv=8, d=128, ctx=4096, ragged=0, page=64,
             window=0, sink=0, layout="hnd"),
        # A server's batch at very different lengths, small pages, token-major pages.
        dict(name="decode_ragged_48", op="decode", batch=48, hq=32, hkv=8, d=128, ctx=16384, ragged=1, page=16,
             window=0, sink=0, layout="nhd"),
        # Sliding-window layers (32 heads of 80, window 4096, sinks) deep into 16K contexts.
        dict(name="decode_window_32", op="decode", batch=32, hq=32, hkv=32, d=80, ctx=16384, ragged=1, page=32,
             window=4096, sink=4, layout="hnd"),
        # The first token after the 1M-token prefill (32 query and 8 KV heads).
        dict(name="decode_one_1m", op="decode", batch=1, hq=32, hkv=8, d=128, ctx=1 << 20, ragged=0, page=128,
             window=0, sink=0, layout="hnd"),
        # A decode step's append: one token for each of 64 sequences, queries rotated along.
        dict(name="append_step_64", op="append", batch=64, hq=32, hkv=8, d=128, ctx=4096, new=1, page=16,
             rot=128, inter=0, norm=1, layout="nhd"),
        # A chunked prefill's append: ragged chunks of four sequences, partial rotation.
        dict(name="append_chunk_4", op="append", batch=4, hq=32, hkv=32, d=80, ctx=16384, new=4096, page=64,
             rot=32, inter=0, norm=0, layout="hnd"),
        # The queries and keys of the 32K GQA prefill before its attention.
        dict(name="qknr_prefill_32k", op="qknr", bwd=0, batch=1, hq=32, hkv=8, n=32768, d=128, rot=128,
             inter=0, norm=1, given=0),
        # The backward of the same pass in a training step of two packed 8K sequences with
        # their own positions, adjacent pairs rotated.
        dict(name="qknr_train_8k", op="qknr", bwd=1, batch=2, hq=32, hkv=8, n=8191, d=128, rot=64,
             inter=1, norm=1, given=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["swa", "swa", "decode", "decode", "append", "qknr"])
    d = rng.choice([64, 80, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 1, 2, 3, 4, 8])
    if op == "swa":
        train = rng.randint(0, 1)
        batch = rng.choice([1, 1, 2, 3])
        n = _log(rng, 1, 16384)
        nk = n if train or rng.random() < 0.5 else n + _log(rng, 1, 4096)
        window = _log(rng, 1, 4096)
        sink = rng.choice([0, 1, 4, 4, rng.randint(1, 300)])
        c = dict(op=op, train=train, batch=batch, hq=hq, hkv=hkv, n=n, nk=nk, d=d, window=window, sink=sink)
        # No dearer than the largest listed one, in pairs and in rows.
        while work(c)["flops"] > 2e12 or c["batch"] * c["hq"] * c["n"] > 32 * 16384:
            c["n"] = (c["n"] + 1) // 2
            c["nk"] = c["n"] if train else max(c["n"], c["nk"] // 2)
        return c
    if op == "decode":
        batch = _log(rng, 1, 128)
        ctx = _log(rng, 1, 262144)
        window = rng.choice([0, 0, _log(rng, 1, 8192)])
        sink = rng.choice([0, 4, rng.randint(1, 200)]) if window else 0
        c = dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, ctx=ctx, ragged=rng.randint(0, 1),
                 page=rng.choice([1, 16, 32, 48, 64, 128, 256]), window=window, sink=sink,
                 layout=rng.choice(["hnd", "nhd"]))
        while c["batch"] * c["hkv"] * c["ctx"] * c["d"] > 8 * 128 * (1 << 19):
            c["ctx"] = (c["ctx"] + 1) // 2
        return c
    rot = rng.choice([r for r in range(16, d + 1, 16)])
    if op == "append":
        batch = _log(rng, 1, 128)
        new = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 16384 // batch))
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, ctx=new + _log(rng, 1, 4096), new=new,
                    page=rng.choice([1, 16, 32, 48, 64, 128, 256]), rot=rot, inter=rng.randint(0, 1),
                    norm=rng.randint(0, 1), layout=rng.choice(["hnd", "nhd"]))
    c = dict(op=op, bwd=rng.randint(0, 1), batch=rng.choice([1, 1, 2, 5]), hq=hq, hkv=hkv, n=_log(rng, 1, 32768),
             d=d, rot=rot, inter=rng.randint(0, 1), norm=rng.randint(0, 1), given=rng.randint(0, 1))
    while c["batch"] * (c["hq"] + c["hkv"]) * c["n"] * c["d"] > 40 * 32768 * 128:
        c["n"] = (c["n"] + 1) // 2
    return c


def _lens(case):
    """Lengths of the sequences, of the case alone: all ``ctx`` tokens, or spread over
    [0, ctx] by their logarithm with the longest among them."""
    r = random.Random(case["batch"] * 1000003 + case["ctx"])
    if not case.get("ragged", 1):
        return [case["ctx"]] * case["batch"]
    ls = [_log(r, 1, case["ctx"] + 1) - 1 for _ in range(case["batch"])]
    ls[r.randrange(len(ls))] = case["ctx"]
    return ls


def _news(case):
    """append: (new tokens, length with them) of every sequence."""
    r = random.Random(case["batch"] * 7919 + case["ctx"] + case["new"])
    if case["new"] == 1:
        news = [1] * case["batch"]
    else:
        news = [r.randint(0, case["new"]) for _ in range(case["batch"])]
        news[r.randrange(len(news))] = case["new"]
    return news, [n + r.randint(0, case["ctx"] - n) for n in news]


def _pairs(n, nk, window, sink):
    """(query, key) pairs of one head: row i at position p = nk - n + i attends the keys
    j <= p with p - j < window or j < sink."""
    def below(m):          # pairs of the first m positions
        w = min(m, window)
        band = w * (w + 1) // 2 + (m - w) * window
        s = min(sink, max(0, m - window))
        return band + s * (s + 1) // 2 + (max(0, m - window) - s) * sink
    return below(nk) - below(nk - n)


def work(case):
    op, d, hq, hkv, b = case["op"], case["d"], case["hq"], case["hkv"], case["batch"]
    if op == "swa":
        n, nk = case["n"], case["nk"]
        pairs = b * hq * _pairs(n, nk, case["window"], case["sink"])
        rows, keys = b * hq * n * d * 2, b * hkv * nk * d * 2
        if not case["train"]:
            return {"bytes": 2 * rows + 2 * keys + b * hq * n * 4, "flops": 4 * d * pairs}
        # Forward, and the five products of the backward; q, dout in, out, lse, dq out;
        # k, v in, dk, dv out.
        return {"bytes": 4 * rows + 4 * keys + b * hq * n * 4, "flops": 14 * d * pairs}
    if op == "decode":
        w = case["window"]
        seen = sum(m if not w else min(m, w) + min(case["sink"], max(0, m - w)) for m in _lens(case))
        return {"bytes": seen * hkv * d * 4 + b * hq * (4 * d + 4), "flops": 4 * d * hq * seen}
    if op == "append":
        t = sum(_news(case)[0])
        heads = hq + 2 * hkv
        return {"bytes": t * heads * d * 4 + t * case["rot"] * 4, "flops": t * (hq + hkv) * (3 * case["rot"] + 4 * d * case["norm"])}
    rows = b * (hq + hkv) * case["n"]
    each = 6 if case["bwd"] and case["norm"] else 4
    tab = case["n"] * case["rot"] * 4
    return {"bytes": rows * d * each + tab, "flops": rows * (3 * case["rot"] + (14 if case["bwd"] else 4) * d * case["norm"])}


# ------------------------------------------------------------------ inputs

def _tables(positions, rot, theta=1e6):
    """cos and sin of position * theta^(-2 i / rot), from 64-bit angles."""
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return a.cos().float(), a.sin().float()


def _pages(case, lens, g, cpu, fill):
    """A cache whose sequences own scattered pages: k, v [pages, hkv, page, d] (in memory
    head-major or token-major), and the table [batch, pages of the longest]."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    need = [-(-m // page) for m in lens]
    total = sum(need) + 3
    shape = (total, hkv, page, d) if case["layout"] == "hnd" else (total, page, hkv, d)
    kv = []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        for a in range(0, total, 4096):
            part = x[a:a + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda") if fill else torch.zeros((), device="cuda"))
        kv.append(x if case["layout"] == "hnd" else x.permute(0, 2, 1, 3))
    perm = torch.randperm(total, generator=cpu, dtype=torch.int32)
    table = torch.zeros(len(lens), max(1, max(need)), dtype=torch.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = perm[at:at + m]
        at += m
    return kv[0], kv[1], table.cuda()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    s = dict(case)
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    if case["op"] == "swa":
        s["q"] = randn(b, hq, case["n"], d, scale=1.5)
        s["k"], s["v"] = randn(b, hkv, case["nk"], d), randn(b, hkv, case["nk"], d)
        if case["train"]:
            s["dout"] = randn(b, hq, case["n"], d)
        return s
    if case["op"] == "decode":
        lens = _lens(case)
        s["k"], s["v"], s["table"] = _pages(case, lens, g, cpu, True)
        s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["longest"] = max(lens)
        s["q"] = randn(b, hq, d, scale=1.5)
        return s
    if case["norm"]:
        s["q_weight"] = randn(d, scale=0.2) + 1
        s["k_weight"] = randn(d, scale=0.2) + 1
    else:
        s["q_weight"] = s["k_weight"] = None
    if case["op"] == "append":
        news, lens = _news(case)
        s["k_pages"], s["v_pages"], s["table"] = _pages(case, lens, g, cpu, False)
        s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        cu = [0]
        for m in news:
            cu.append(cu[-1] + m)
        s["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
        s["cos"], s["sin"] = _tables(case["ctx"], case["rot"])
        # The three projections of a token lie beside each other.
        qkv = randn(cu[-1], hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = qkv.split([hq, hkv, hkv], 1)
        return s
    n = case["n"]
    x = randn(b, n, hq + hkv, d).permute(0, 2, 1, 3)
    s["q"], s["k"] = x[:, :hq], x[:, hq:]
    s["cos"], s["sin"] = _tables(n, case["rot"])
    s["positions"] = None
    if case["given"]:
        # Packed sequences: positions that start again.
        cut = torch.randint(1, n + 1, (b, 1), generator=cpu)
        at = torch.arange(n)[None]
        s["positions"] = torch.where(at < cut, at, at - cut).to(torch.int32).cuda()
    if case["bwd"]:
        s["dq_out"], s["dk_out"] = randn(b, hq, n, d), randn(b, hkv, n, d)
    return s


# ------------------------------------------------------------------ the operators

def run(s):
    return {"swa": _swa, "decode": _decode, "append": _append, "qknr": _qknr}[s["op"]](s)


def _swa(s):
    q, k, v, window, sink = s["q"], s["k"], s["v"], s["window"], s["sink"]
    if own:
        import block_sparse_long_prefill_b200 as moba
        out, lse = moba.swa_attn_fwd_chunk(q, k, v, window, sink=sink)
        if not s["train"]:
            return {"out": out, "lse": lse}
        dq, dk, dv = moba.swa_attn_bwd(q, k, v, out, lse, s["dout"], window, sink=sink)
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    b, hq, n, d = q.shape
    hkv, nk = k.shape[1:3]
    G, scale = hq // hkv, d ** -0.5
    # Query blocks of C rows against the C + window - 1 keys that any of them reaches and,
    # in columns of their own, the sinks.
    C = min(1024, n)
    nb = -(-n // C)
    first = min(sink, nk)
    back = min(window - 1, nk - 1)
    pos = nk - n + torch.arange(nb * C, device="cuda").view(nb, C, 1)
    key = pos[:, :1, 0] - back + torch.arange(C + back, device="cuda")                   # [nb, C + back]
    band = (key[:, None] <= pos) & (pos - key[:, None] < window) & (key[:, None] >= first) & (key[:, None] < nk)
    at = torch.cat([torch.arange(first, device="cuda").expand(nb, first), key.clamp(0, nk - 1)], 1)
    see = torch.cat([torch.arange(first, device="cuda") <= pos, band], 2)[:, None]        # [nb, 1, C, cols]

    def rows(x):
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, nb * C - n))
        return x.view(b, hkv, G, nb, C, d).transpose(2, 3).reshape(b, hkv, nb, G * C, d)

    def back_rows(x):
        return x.view(b, hkv, nb, G, C, -1).transpose(2, 3).reshape(b, hq, nb * C, -1)[:, :, :n]

    qf, kf, vf = rows(q), k.float()[:, :, at], v.float()[:, :, at]
    z = (qf @ kf.transpose(-1, -2)).mul_(scale).view(b, hkv, nb, G, C, -1).masked_fill_(~see, -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-1e30)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(total.clamp_min(1e-30)).view(b, hkv, nb, G * C, -1)
    out = p @ vf
    lse = back_rows(total.log() + top)[..., 0]
    res = {"out": back_rows(out).to(q.dtype), "lse": lse}
    if not s["train"]:
        return res
    g = rows(s["dout"])
    dvf = p.transpose(-1, -2) @ g
    dz = (g @ vf.transpose(-1, -2)).sub_((g * out).sum(-1, keepdim=True)).mul_(p)
    dkf = (dz.transpose(-1, -2) @ qf).mul_(scale)
    res["dq"] = back_rows((dz @ kf).mul_(scale)).to(q.dtype)

    def to_keys(x):
        return torch.zeros(b, hkv, nk, d, device="cuda").index_add_(2, at.reshape(-1), x.reshape(b, hkv, -1, d))

    res["dk"], res["dv"] = to_keys(dkf).to(k.dtype), to_keys(dvf).to(v.dtype)
    return res


def _decode(s):
    q, kp, vp, table, lens = s["q"], s["k"], s["v"], s["table"], s["lens"]
    if own:
        import block_sparse_long_prefill_b200 as moba
        out, lse = moba.paged_decode_attn(q, kp, vp, table, lens, window=s["window"], sink=s["sink"])
        return {"out": out, "lse": lse}
    b, hq, d = q.shape
    hkv, page = kp.shape[1:3]
    j = torch.arange(s["longest"], device="cuda")
    pid, slot = table.long()[:, j // page], (j % page).expand(b, -1)
    kf = kp[pid, :, slot].float().transpose(1, 2)                                         # [b, hkv, keys, d]
    z = (q.float().view(b, hkv, -1, d) @ kf.transpose(-1, -2)).mul_(d ** -0.5)
    del kf
    n = lens.long()[:, None]
    see = j < n
    if s["window"]:
        see = see & ((n - 1 - j < s["window"]) | (j < s["sink"]))
    z = z.masked_fill_(~see[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-1e30) if s["longest"] else z.new_zeros(b, hkv, hq // hkv, 1)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ vp[pid, :, slot].float().transpose(1, 2)) / total.clamp_min(1e-30)
    return {"out": out.view(b, hq, d).to(q.dtype), "lse": (total.log() + top).view(b, hq)}


def _norm(x, w):
    x = x.float()
    if w is None:
        return x
    return x * (x.square().mean(-1, keepdim=True) + _EPS).rsqrt() * w.float()


def _turn(x, cos, sin, inter):
    """The first 2 * cos.shape[-1] columns of x turned by the angles: pairs of neighbours
    (inter), or of the two halves."""
    h = cos.shape[-1]
    y = x[..., :2 * h]
    a, c = (y[..., 0::2], y[..., 1::2]) if inter else (y[..., :h], y[..., h:])
    u, w = a * cos - c * sin, c * cos + a * sin
    y = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([y, x[..., 2 * h:]], -1)


def _append(s):
    q, k, v, cu, lens = s["q"], s["k"], s["v"], s["cu"], s["lens"]
    if own:
        import block_sparse_long_prefill_b200 as moba
        q_out = moba.kv_append(k, v, s["k_pages"], s["v_pages"], s["table"], lens,
                               cu_seqlens=None if s["new"] == 1 else cu, cos=s["cos"], sin=s["sin"],
                               k_weight=s["k_weight"], q=q, q_weight=s["q_weight"], eps=_EPS,
                               interleaved=bool(s["inter"]))
        return {"q_out": q_out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    t = torch.arange(k.shape[0], device="cuda")
    seq = torch.searchsorted(cu.long(), t, right=True) - 1
    pos = lens.long()[seq] - cu.long()[seq + 1] + t
    page = s["k_pages"].shape[2]
    pid, slot = s["table"].long()[seq, pos // page], pos % page
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q_out = _turn(_norm(q, s["q_weight"]), cos, sin, s["inter"]).to(q.dtype)
    s["k_pages"][pid, :, slot] = _turn(_norm(k, s["k_weight"]), cos, sin, s["inter"]).to(k.dtype)
    s["v_pages"][pid, :, slot] = v
    return {"q_out": q_out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _qknr(s):
    q, k, qw, kw = s["q"], s["k"], s["q_weight"], s["k_weight"]
    if own:
        import block_sparse_long_prefill_b200 as moba
        how = dict(positions=s["positions"], q_weight=qw, k_weight=kw, eps=_EPS, interleaved=bool(s["inter"]))
        if not s["bwd"]:
            q_out, k_out = moba.qk_norm_rope_fwd(q, k, s["cos"], s["sin"], **how)
            return {"q_out": q_out, "k_out": k_out}
        dq, dk, dqw, dkw = moba.qk_norm_rope_bwd(s["dq_out"], s["dk_out"], q, k, s["cos"], s["sin"], **how)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    cos, sin = s["cos"], s["sin"]
    if s["positions"] is not None:
        cos, sin = cos[s["positions"].long()][:, None], sin[s["positions"].long()][:, None]
    if not s["bwd"]:
        return {"q_out": _turn(_norm(q, qw), cos, sin, s["inter"]).to(q.dtype),
                "k_out": _turn(_norm(k, kw), cos, sin, s["inter"]).to(k.dtype)}
    dq, dqw = _qknr_back(s["dq_out"], q, qw, cos, sin, s["inter"])
    dk, dkw = _qknr_back(s["dk_out"], k, kw, cos, sin, s["inter"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _qknr_back(dy, x, w, cos, sin, inter):
    g = _turn(dy.float(), cos, -sin, inter)
    if w is None:
        return g.to(x.dtype), None
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + _EPS).rsqrt()
    xn = x * r
    dw = (g * xn).sum((0, 1, 2))
    g = g * w.float()
    return ((g - xn * (g * xn).mean(-1, keepdim=True)) * r).to(dy.dtype), dw


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"swa": _exact_swa, "decode": _exact_decode, "append": _exact_append, "qknr": _exact_qknr}[case["op"]](s)


def _exact_swa(s):
    q, k, v = s["q"], s["k"], s["v"]
    b, hq, n, d = q.shape
    nk, G, f64 = k.shape[2], hq // k.shape[1], torch.float64
    names = ["out", "dq"] if s["train"] else ["out"]
    res = {m: torch.zeros(q.shape, dtype=f64, device="cuda") for m in names}
    res["lse"] = torch.zeros(b, hq, n, dtype=f64, device="cuda")
    if s["train"]:
        res["dk"], res["dv"] = (torch.zeros(k.shape, dtype=f64, device="cuda") for _ in range(2))
    for i in range(b):
        for h in range(hq):
            kk, vv = k[i, h // G].double(), v[i, h // G].double()
            for a in range(0, n, 2048):
                e = min(n, a + 2048)
                p = torch.arange(nk - n + a, nk - n + e, device="cuda")[:, None]
                hi = nk - n + e
                j = torch.arange(hi, device="cuda")
                hide = (j > p) | ((p - j >= s["window"]) & (j >= s["sink"]))
                qq = q[i, h, a:e].double()
                z = (qq @ kk[:hi].T / math.sqrt(d)).masked_fill_(hide, -math.inf)
                lse = torch.logsumexp(z, -1)
                w = torch.exp(z - lse[:, None])
                o = w @ vv[:hi]
                res["out"][i, h, a:e], res["lse"][i, h, a:e] = o, lse
                if s["train"]:
                    go = s["dout"][i, h, a:e].double()
                    gz = w * (go @ vv[:hi].T - (go * o).sum(-1, keepdim=True)) / math.sqrt(d)
                    res["dq"][i, h, a:e] = gz @ kk[:hi]
                    res["dk"][i, h // G, :hi] += gz.T @ qq
                    res["dv"][i, h // G, :hi] += w.T @ go
    return res


def _exact_decode(s):
    q, page = s["q"].double(), s["k"].shape[2]
    b, hq, d = q.shape
    hkv = s["k"].shape[1]
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        own_pages = s["table"][i, :-(-n // page)].long()
        j = torch.arange(n, device="cuda")
        kept = (n - 1 - j < s["window"]) | (j < s["sink"]) | (s["window"] == 0)
        for h in range(hkv):
            kk = s["k"][own_pages, h].reshape(-1, d)[:n][kept].double()
            vv = s["v"][own_pages, h].reshape(-1, d)[:n][kept].double()
            mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            z = q[i, mine] @ kk.T / math.sqrt(d)
            lse[i, mine] = torch.logsumexp(z, -1)
            out[i, mine] = torch.softmax(z, -1) @ vv
    return {"out": out, "lse": lse}


def _exact_turned(x, w, pos, cos, sin, inter, sign=1.0):
    """x [..., d] at positions pos [...] by complex products: pair (a, c) -> (a + ic) e^(i angle)."""
    x = x.double()
    d, h = x.shape[-1], cos.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + _EPS) * w.double()
    i = torch.arange(h, device="cuda")
    ia, ic = (2 * i, 2 * i + 1) if inter else (i, i + h)
    turned = torch.complex(x[..., ia], x[..., ic]) * torch.complex(cos[pos].double(), sign * sin[pos].double())
    y = x.clone()
    y[..., ia], y[..., ic] = turned.real, turned.imag
    return y


def _exact_append(s):
    lens, cu, page = s["lens"].tolist(), s["cu"].tolist(), s["k_pages"].shape[2]
    pos = [lens[i] - (cu[i + 1] - cu[i]) + r for i in range(len(lens)) for r in range(cu[i + 1] - cu[i])]
    seq = [i for i in range(len(lens)) for _ in range(cu[i + 1] - cu[i])]
    pos, seq = torch.tensor(pos, device="cuda"), torch.tensor(seq, device="cuda")
    at = pos[:, None]
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    pid = s["table"].long()[seq, pos // page]
    kp[pid, :, pos % page] = _exact_turned(s["k"], s["k_weight"], at, s["cos"], s["sin"], s["inter"])
    vp[pid, :, pos % page] = s["v"].double()
    return {"q_out": _exact_turned(s["q"], s["q_weight"], at, s["cos"], s["sin"], s["inter"]),
            "k_pages": kp, "v_pages": vp}


def _exact_qknr(s):
    b, n = s["q"].shape[0], s["q"].shape[2]
    pos = torch.arange(n, device="cuda").expand(b, n) if s["positions"] is None else s["positions"].long()
    pos = pos[:, None]
    if not s["bwd"]:
        return {"q_out": _exact_turned(s["q"], s["q_weight"], pos, s["cos"], s["sin"], s["inter"]),
                "k_out": _exact_turned(s["k"], s["k_weight"], pos, s["cos"], s["sin"], s["inter"])}
    res = {}
    for m in "qk":
        w, x = s[m + "_weight"], s[m].double()
        g = _exact_turned(s["d%s_out" % m], None, pos, s["cos"], s["sin"], s["inter"], -1.0)
        if w is None:
            res["d" + m], res["d%s_weight" % m] = g, None
            continue
        ms = (x * x).mean(-1, keepdim=True) + _EPS
        res["d%s_weight" % m] = (g * x / torch.sqrt(ms)).sum((0, 1, 2))
        gw = g * w.double()
        res["d" + m] = gw / torch.sqrt(ms) - x * (gw * x).mean(-1, keepdim=True) / ms ** 1.5
    return res
