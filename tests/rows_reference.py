"""Plain 64-bit references of the row append and the attentions, and the error
bounds their results are held to."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half of the smallest step: values below the normal range
FLOOR = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def rotated(x, positions, inv_freq, start, interleaved, sections):
    """x [T, heads, dim] in float64, rotated pair by pair."""
    y = x.double().clone()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    half = len(axis)
    for i in range(half):
        ang = positions[axis[i]].double() * inv_freq[i].double()
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        a, b = (start + 2 * i, start + 2 * i + 1) if interleaved else \
            (start + i, start + half + i)
        p, q = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = p * c - q * s, q * c + p * s
    return y


def rotation_bound(want, x, dtype):
    """One rounding to the type, and fp32 inside: the turn's fraction is off by
    2^-26, its sine and cosine by 2^-22 in all, the two products and the sum by
    2^-24 each, of at most the head's largest two values."""
    return HALF_STEP[dtype] * want.abs() + FLOOR[dtype] + \
        2.0 ** -20 * 2 * x.double().abs().amax(-1, keepdim=True)


def attention(q, keys, values, positions, window, sinks, scale):
    """q [n, hq, kd]; keys [nk, hkv, kd], values [nk, hkv, vd] of one request, query
    i at positions[i].  Returns out, lse and the error bound of out, float64.

    Bound: a score is off by at most kd 2^-24 sum |q k| scale (fp32 sums in any
    order) and 2^-22 relative of itself (its scaling and the exponential), so a
    weight by d = twice that; weights are rounded to the type up to twice; fp32
    sums add 2^-20; the result is rounded once."""
    n, hq, kd = q.shape
    nk, hkv, _ = keys.shape
    g = hq // hkv
    dtype = q.dtype
    at = torch.arange(nk, device=q.device)
    pos = positions[:, None]
    see = at[None] <= pos
    if window:
        see &= (pos - at[None] < window) | (at[None] < sinks)
    out = torch.zeros(n, hq, values.shape[2], dtype=torch.float64, device=q.device)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    if nk == 0 or n == 0:
        return out, lse, bound, lse_bound
    for h in range(hq):
        k, v = keys[:, h // g].double(), values[:, h // g].double()
        x = q[:, h].double()
        s = (x @ k.t().contiguous()) * scale
        size = (x.abs() @ k.abs().t().contiguous()) * scale
        s = s.masked_fill(~see, -math.inf)
        size = size.masked_fill(~see, 0.0)
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
        p = p.masked_fill(~see, 0.0)
        lse[:, h] = z
        # rows of a masked key that hold infinities or NaN count for nothing
        vv = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
        out[:, h] = p @ vv
        for j in torch.nonzero(~torch.isfinite(v).all(1)).flatten().tolist():
            rows = see[:, j]
            out[rows, h] += p[rows, j, None] * (v[j] - vv[j])
        d = 2 * (kd * 2.0 ** -24 * size.amax(1) + 2.0 ** -22 * s.masked_fill(~see, 0).abs().amax(1))
        size_out = p @ vv.abs()
        bound[:, h] = HALF_STEP[dtype] * out[:, h].abs() + FLOOR[dtype] + \
            (2 * HALF_STEP[dtype] + 2 * d[:, None] + 2.0 ** -20) * size_out
        lse_bound[:, h] = d + 2.0 ** -20 * (1 + torch.where(z == -math.inf, 0 * z, z.abs()))
    return out, lse, bound, lse_bound


def check(out, lse, want):
    """Every value within its bound; what has no finite value has to agree."""
    w_out, w_lse, bound, lse_bound = want
    o = out.double()
    fin = torch.isfinite(w_out)
    assert torch.equal(torch.isfinite(o), fin), "finite where it should not be, or the reverse"
    err = (o - w_out).abs().masked_fill(~fin, 0.0) - bound.masked_fill(~fin, 1.0)
    assert err.max() <= 0, "out off its bound by %g" % float(err.max())
    if lse is not None:
        gone = w_lse == -math.inf
        assert torch.equal(lse == -math.inf, gone)
        ok = torch.isfinite(w_lse)
        e = (lse.double() - w_lse).abs()[ok] - lse_bound[ok]
        assert e.numel() == 0 or e.max() <= 0, "lse off its bound by %g" % float(e.max())
