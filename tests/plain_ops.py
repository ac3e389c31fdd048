"""Plain formulations in float64 of the operators around the attention kernels, written
from their formulas, with the bounds that the kernels' roundings allow.

Bounds count half steps: a value rounded to bf16 is off by at most 2^-8 of itself, one
rounded to float32 by 2^-24.  The kernels compute in float32 and round to bf16 where a
result is stored and where a probability or dz enters a tensor-core product; ``SLACK``
covers what the bounds leave out: the float32 sums (at most a few thousand terms of 2^-24
each, below 2^-11 of the sums of magnitudes, an eighth of 2^-8) and products of two
roundings (2^-8 of the bound)."""
import math

import torch

BF16, F32 = 2.0 ** -8, 2.0 ** -24
SLACK = 1.125 + 2.0 ** -8
# A probability below 2^-126 is flushed to zero, in float32's exponential and in bf16: that
# moves a dz by at most 2^-126 (|dp| + |D|), and with magnitudes below 2^10 a sum of 2^12
# products of such dz with q or k by less than 2^-126 2^12 2^10 2^12 = 2^-92.
FLUSH = 2.0 ** -92


def visible(nq, nk, window, sink, device="cpu"):
    """[nq, nk] truth: row i at position nk - nq + i sees keys j <= p, p - j < window or
    j < sink (window 0: no limit)."""
    p = torch.arange(nk - nq, nk, device=device)[:, None]
    j = torch.arange(nk, device=device)[None]
    near = (p - j < window) if window else torch.ones_like(j <= p)
    return (j <= p) & (near | (j < sink))


def attention(q, k, v, see, scale=None):
    """q [.., nq, d], k, v [.., nk, d] float64; returns out, lse, p and the bound of out."""
    scale = scale or q.shape[-1] ** -0.5
    z = (q @ k.transpose(-1, -2) * scale).masked_fill(~see, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.where(see, torch.exp(z - torch.nan_to_num(lse, neginf=0.0)[..., None]), 0.0)
    out = p @ v
    # P rounded to bf16 against V, and the stored result.
    bound = SLACK * BF16 * (out.abs() + p @ v.abs()) + FLUSH
    # A score is a float32 sum of d products.
    zerr = (q.shape[-1] + 8) * F32 * scale * (q.abs() @ k.abs().transpose(-1, -2)).amax(-1)
    lse_bound = zerr + 2.0 ** -19 * lse.abs().nan_to_num(posinf=0.0).clamp_min(1.0)
    return out, lse, p, bound, lse_bound


def attention_bwd(q, k, v, do, see, scale=None, out_bound=None):
    """Gradients and their bounds; out_bound: how far the `out` that the kernel is given may
    be from the formula's (default: its rounding to bf16)."""
    scale = scale or q.shape[-1] ** -0.5
    out, lse, p, _, _ = attention(q, k, v, see, scale)
    if out_bound is None:
        out_bound = BF16 * out.abs()
    dsum = (do * out).sum(-1, keepdim=True)
    derr = (do.abs() * out_bound).sum(-1, keepdim=True)
    dz = p * (do @ v.transpose(-1, -2) - dsum)
    dzerr = BF16 * dz.abs() + p * derr
    dq, dk, dv = scale * dz @ k, scale * dz.transpose(-1, -2) @ q, p.transpose(-1, -2) @ do
    bq = SLACK * (BF16 * dq.abs() + scale * dzerr @ k.abs())
    bk = SLACK * (BF16 * dk.abs() + scale * dzerr.transpose(-1, -2) @ q.abs())
    bv = SLACK * (BF16 * dv.abs() + BF16 * p.transpose(-1, -2) @ do.abs())
    # float32 scores (|z| up to a few tens) move every p, dz and their sums.
    slack = 2.0 ** -13 * SLACK
    bq = bq + slack * scale * (p * ((do @ v.transpose(-1, -2)).abs() + dsum.abs())) @ k.abs()
    bk = bk + slack * scale * (p * ((do @ v.transpose(-1, -2)).abs() + dsum.abs())).transpose(-1, -2) @ q.abs()
    return (dq, bq + FLUSH), (dk, bk + FLUSH), (dv, bv + FLUSH)


def attention_bwd_norms(q, k, v, do, see, scale=None):
    """How far the kernels' whole gradients may be from the formula's, in the 2-norm (dq, dk, dv).

    Roundings to bf16 err by at most 2^-8 of the value and, value by value, with independent
    signs, so their squares add up: of the stored result, of each dz (of each P for dv), and,
    through D = dO.o, of the stored ``out`` and of the P behind it.  (Each is at its largest
    here; a rounding's root mean square is less than half of it, which leaves room for the
    float32 sums.)"""
    scale = scale or q.shape[-1] ** -0.5
    out, _, p, _, _ = attention(q, k, v, see, scale)
    dp = do @ v.transpose(-1, -2)
    dz = p * (dp - (do * out).sum(-1, keepdim=True))
    dq, dk, dv = scale * dz @ k, scale * dz.transpose(-1, -2) @ q, p.transpose(-1, -2) @ do
    derr2 = (do.square() * out.square()).sum(-1, keepdim=True) + (p * dp).square().sum(-1, keepdim=True)
    dqn = dq.square().sum() + scale ** 2 * ((dz.square() @ k.square()).sum() + (derr2 * (p @ k).square()).sum())
    # (A row's error in D reaches every key that it sees.)
    dkn = dk.square().sum() + scale ** 2 * ((dz.square().transpose(-1, -2) @ q.square()).sum()
                                            + (p.square().transpose(-1, -2) @ (derr2 * q.square())).sum())
    dvn = dv.square().sum() + (p.square().transpose(-1, -2) @ do.square()).sum()
    return tuple(BF16 * float(x) ** 0.5 for x in (dqn, dkn, dvn))


def turn(x, cos, sin, interleaved, sign=1.0):
    """Rotation of the first 2 * cos.shape[-1] columns; returns the result and the sum of
    magnitudes behind each value."""
    h = cos.shape[-1]
    i = torch.arange(h, device=x.device)
    ia, ic = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    y, mag = x.clone(), x.abs().clone()
    a, c, s = x[..., ia], x[..., ic], sign * sin
    y[..., ia], y[..., ic] = a * cos - c * s, c * cos + a * s
    mag[..., ia], mag[..., ic] = (a * cos).abs() + (c * s).abs(), (c * cos).abs() + (a * s).abs()
    return y, mag


def norm_rope(x, w, cos, sin, interleaved, eps):
    """x [.., d] float64, cos, sin [.., rot / 2] of its positions.  Bound: the stored result
    and float32 arithmetic (the mean of squares, a root, four products: 2^-20 of the terms)."""
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    y, mag = turn(x, cos, sin, interleaved)
    return y, BF16 * y.abs() + 2.0 ** -20 * mag + 1e-38


def norm_rope_bwd(dy, x, w, cos, sin, interleaved, eps):
    """Returns dx with its bound, and dw [d] with its (None without a weight)."""
    g, gmag = turn(dy, cos, sin, interleaved, -1.0)
    if w is None:
        return (g, BF16 * g.abs() + 2.0 ** -20 * gmag + 1e-38), None
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    gw = g * w
    m = (gw * x).mean(-1, keepdim=True) * r ** 2
    dx = r * (gw - x * m)
    mmag = (gmag * w.abs() * x.abs()).mean(-1, keepdim=True) * r ** 2
    bound = BF16 * dx.abs() + 2.0 ** -19 * r * (gmag * w.abs() + x.abs() * mmag) + 1e-38
    dims = tuple(range(dy.dim() - 1))
    dw = (g * x * r).sum(dims)
    # A lane's run, the CTA's lanes and the CTAs: fewer than 512 float32 additions deep.
    return (dx, bound), (dw, 512 * F32 * (gmag * x.abs() * r).sum(dims) + 1e-38)


def gather_pages(pages, table, n):
    """The first n positions of a sequence: pages [P, hkv, page, d] -> [hkv, n, d] float64."""
    page = pages.shape[2]
    own = table[:-(-n // page)].long()
    x = pages[own].double().transpose(0, 1).reshape(pages.shape[1], -1, pages.shape[3])
    return x[:, :n]


def check(name, got, want, bound):
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        over = ((got - want).abs() / bound.clamp_min(1e-300)).nan_to_num(nan=math.inf)
        at = int(over.flatten().argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values off; worst {float(over.max()):.3g} "
                             f"bounds at {at}: {got.flatten()[at]} for {want.flatten()[at]}")
