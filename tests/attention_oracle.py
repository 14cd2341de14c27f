"""Plain 64-bit forms of the attention operators (norms of queries and keys
with the rotation, attention with a window, first tokens and a bias by buckets)
and the bounds their kernels are held to.  torch on the CPU, written from the
formulas; nothing here comes from the HIP path.

Bounds.  u = 2^-24 is half a step of binary32, u_t half a step of the stored
type.  A binary32 sum of n terms is off by at most 2 n u times the sum of the
magnitudes, whatever its order and whether an addition rounds or cuts off (a
matrix unit's may).  A score so is off by
  e_s = 2 (dim + 4) u scale sum|q||k| + 4 u (|s| + |bias|),
and a weight exp(s - m) relatively by e_s, the roundings of the difference
(4 u |s - m|) and of the exponential itself (8 u: a few steps).  Weights are
rounded to the element type (u_t relatively; binary16 below 2^-14 by 2^-25),
and so is ds, for binary16 in units of at most twice the largest |do_i| of the
rows that meet in a sum.  First order throughout, with 1 % for the rest.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def stored(bound, value, dtype):
    """The bound after the value is rounded to its stored type."""
    return 1.01 * bound + HALF[dtype] * (value.abs() + bound) + TINY[dtype]


# ---- norms of queries and keys, rotation ------------------------------------------------

def angles(positions, rot, base):
    """positions x rot / 2 x (cos, sin) in 64 bits."""
    p = torch.arange(rot // 2, dtype=torch.float64)
    a = torch.as_tensor(positions, dtype=torch.float64)[:, None] * base ** (-2.0 * p / max(rot, 1))
    return torch.stack([a.cos(), a.sin()], 2)


def turned(u, cs, interleaved, back=False):
    """u (tokens, heads, dim) turned by cs (tokens, rot / 2, 2)."""
    rot = 2 * cs.shape[1]
    out = u.clone()
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * (-1.0 if back else 1.0)
    out[..., a] = u[..., a] * c - u[..., b] * s
    out[..., b] = u[..., b] * c + u[..., a] * s
    return out


def _spread(e, cs, interleaved):
    """What an error e of u becomes by the turn: |cos|, |sin| of both of a pair."""
    rot = 2 * cs.shape[1]
    out = e.clone()
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    c, s = cs[:, None, :, 0].abs(), cs[:, None, :, 1].abs()
    out[..., a] = e[..., a] * c + e[..., b] * s
    out[..., b] = e[..., b] * c + e[..., a] * s
    return out


def qk_fwd(x, w, cs, eps, interleaved):
    """(y, bound before the store); x, w, cs in 64 bits; cs None: no rotation."""
    n = x.shape[2]
    rstd = (x.square().mean(2, keepdim=True) + eps).rsqrt()
    u = x * rstd * w
    e = (2 * (n + 4) * U / 2 + 8 * U) * u.abs()            # half of the sum's relative error, and a few roundings
    if cs is None:
        return u, e
    y = turned(u, cs, interleaved)
    return y, _spread(e + 4 * U * u.abs(), cs, interleaved)


def qk_bwd(dy, x, w, cs, eps, interleaved):
    """((dx, dw), bounds before the store)."""
    n = x.shape[2]
    rstd = (x.square().mean(2, keepdim=True) + eps).rsqrt()
    h = x * rstd
    r = (n + 4) * U + 8 * U                                # relative, of rstd and h
    g = dy if cs is None else turned(dy, cs, interleaved, True)
    e_g = torch.zeros_like(dy) if cs is None else _spread(4 * U * dy.abs(), cs, interleaved)
    rows = dy.shape[0] * dy.shape[1]
    dw, e_dw = (g * h).sum((0, 1)), ((e_g + (r + 2 * rows * U) * g.abs()) * h.abs()).sum((0, 1))
    gw, e_gw = g * w, (e_g + U * g.abs()) * w.abs()
    mean = (gw * h).mean(2, keepdim=True)
    e_mean = ((e_gw + (r + (2 * n + 4) * U) * gw.abs()) * h.abs()).mean(2, keepdim=True)
    t = gw - h * mean
    e_t = e_gw + h.abs() * e_mean + (r + 2 * U) * (h * mean).abs() + 2 * U * gw.abs()
    return (rstd * t, dw), (rstd * (e_t + (r + 2 * U) * t.abs()), e_dw)


# ---- attention -----------------------------------------------------------------------------

def bucket(d, starts):
    return torch.bucketize(d, torch.as_tensor(list(starts)), right=True) - 1


def visible(n, window, sinks):
    i = torch.arange(n)
    d = i[:, None] - i[None]
    return (d >= 0) & (((d < window) if window else torch.ones_like(d, dtype=torch.bool)) | (i[None] < sinks))


def _scores(q, k, bias_row, starts, scale, see):
    """One head's scores of one sequence, and their error."""
    n = q.shape[0]
    s = scale * (q @ k.T)
    e = 2 * (q.shape[1] + 4) * U * scale * (q.abs() @ k.abs().T) + 4 * U * s.abs()
    if bias_row is not None:
        d = (torch.arange(n)[:, None] - torch.arange(n)[None]).clamp(min=0)
        b = bias_row[bucket(d, starts)]
        s = s + b
        e = e + 4 * U * (b.abs() + s.abs())
    return s.masked_fill(~see, -math.inf), e.masked_fill(~see, 0.0)


def attention_fwd(q, k, v, bias, starts, scale, window, sinks, edges, dtype):
    """(o, lse) and bounds; o's before the store.  Rows outside the sequences are NaN."""
    t, hq, d = q.shape
    hk = k.shape[1]
    o, e_o = torch.full((t, hq, d), math.nan, dtype=torch.float64), torch.zeros(t, hq, d, dtype=torch.float64)
    lse, e_lse = torch.full((hq, t), math.nan, dtype=torch.float64), torch.zeros(hq, t, dtype=torch.float64)
    for a, b in zip(edges, edges[1:]):
        n = b - a
        if not n:
            continue
        see = visible(n, window, sinks)
        for h in range(hq):
            vv = v[a:b, h * hk // hq]
            s, e = _scores(q[a:b, h], k[a:b, h * hk // hq], None if bias is None else bias[h], starts, scale, see)
            m = s.amax(1, keepdim=True)
            far = (s - m).masked_fill(~see, 0.0).abs()
            r = (e + 4 * U * (far + m.abs()) + 8 * U).masked_fill(~see, 0.0)
            p = torch.exp(s - m)
            total = p.sum(1, keepdim=True)
            p, x = p / total, (r * p).sum(1, keepdim=True) / total + 2 * (n + 8) * U
            y = p @ vv
            o[a:b, h] = y
            e_o[a:b, h] = ((r + HALF[dtype]) * p) @ vv.abs() + (x + 2 * (n + 8) * U) * (p @ vv.abs()) + \
                (2.0 ** -25 * see.double() / total) @ vv.abs() * (dtype == torch.float16)
            lse[h, a:b] = (m + torch.log(total))[:, 0]
            e_lse[h, a:b] = (x + 4 * U * (m.abs() + total.log().abs()) + 8 * U)[:, 0]
    return (o, lse), (e_o, 1.01 * e_lse)


def attention_bwd(do, o, lse, q, k, v, bias, starts, scale, window, sinks, edges, dtype):
    """(dq, dk, dv, dbias) and bounds before the store."""
    t, hq, d = q.shape
    hk = k.shape[1]
    new = lambda *s: torch.zeros(*s, dtype=torch.float64)
    dq, dk, dv = new(t, hq, d), new(t, hk, d), new(t, hk, d)
    e_dq, e_dk, e_dv = new(t, hq, d), new(t, hk, d), new(t, hk, d)
    count = 0 if bias is None else bias.shape[1]
    db, e_db, n_db = new(hq, count), new(hq, count), new(hq, count)
    half, f16 = HALF[dtype], dtype == torch.float16
    for a, b in zip(edges, edges[1:]):
        n = b - a
        if not n:
            continue
        see = visible(n, window, sinks)
        for h in range(hq):
            g = h * hk // hq
            kk, vv, qq, dd, oo = k[a:b, g], v[a:b, g], q[a:b, h], do[a:b, h], o[a:b, h]
            s, e = _scores(qq, kk, None if bias is None else bias[h], starts, scale, see)
            l = lse[h, a:b, None]
            r = (e + 4 * U * ((s - l).masked_fill(~see, 0.0).abs() + l.abs()) + 8 * U).masked_fill(~see, 0.0)
            p = torch.exp(s - l)
            delta = (dd * oo).sum(1, keepdim=True)
            diff = (dd @ vv.T) - delta
            e_diff = 2 * (d + 4) * U * (dd.abs() @ vv.abs().T + (dd * oo).abs().sum(1, keepdim=True)) + 2 * U * diff.abs()
            ds = p * diff
            e_ds = p * (r * diff.abs() + e_diff) + 2 * U * ds.abs()
            norm = dd.square().sum(1, keepdim=True).sqrt()
            # what rounding ds takes: relatively half a step; binary16 at least 2^-25 units of twice the largest |do|
            lost = lambda of: half * (ds.abs() + e_ds) + (2.0 ** -24 * of * see if f16 else 0.0)
            depth = 2 * (n + 8) * U
            dq[a:b, h] = scale * (ds @ kk)
            e_dq[a:b, h] = scale * ((e_ds + lost(norm) + depth * ds.abs()) @ kk.abs())
            # the unit follows the rows as they come: the largest so far is at most the sequence's, of all its heads
            most = do[a:b, g * (hq // hk):(g + 1) * (hq // hk)].square().sum(2).sqrt().max()
            e_k = e_ds + lost(most) + depth * (hq // hk) * ds.abs()
            dk[a:b, g] += scale * (ds.T @ qq)
            e_dk[a:b, g] += scale * (e_k.T @ qq.abs())
            dv[a:b, g] += p.T @ dd
            e_p = p * (r + half + depth * (hq // hk)) + (2.0 ** -31 * see if f16 else 0.0)
            e_dv[a:b, g] += e_p.T @ dd.abs()
            if count:
                idx = bucket((torch.arange(n)[:, None] - torch.arange(n)[None]).clamp(min=0), starts).flatten()
                db[h].index_add_(0, idx, ds.flatten())
                e_db[h].index_add_(0, idx, (e_ds + 2 * U * (n + 300) * ds.abs()).flatten())
    return (dq, dk, dv, db), (e_dq, e_dk, e_dv, e_db)
