"""Measured cases of the attention side of a transformer block: the norms of
queries and keys with the position rotation in the same pass, causal attention
with a sliding window and first tokens that stay visible, and the same with a
learned relative position bias by buckets; forward and backward.

`run` computes a case either in plain torch operations (own = False) or with
the framework's entry points (own = True).

The arithmetic, for packed tokens of one or more sequences (32 bits inside,
rounded once where it is stored):

  qk    for each token and head, over its `dim` elements:
        rstd = 1 / sqrt(mean(x^2) + eps), u = x * rstd * w, and the first
        `rot` elements of u turned in pairs by the token's position:
        (a, b) -> (a cos - b sin, b cos + a sin), the pair p being elements
        (p, p + rot/2), or (2p, 2p + 1) where interleaved;
        backward: g' = dy turned back, h = x * rstd, dw = sum of g' h over
        tokens and heads, g = g' w, dx = rstd * (g - h * mean(g h))
  attn  position j is visible to position i of the same sequence where j <= i
        and (i - j < window or j < sinks); s = scale q.k (+ the bias of the
        head and of the bucket of i - j), p = softmax(s), o = p v,
        lse = log of the sum of exp(s); query head h reads key head
        h // (heads / kv_heads);
        backward, from o and lse: p = exp(s - lse), delta = do.o,
        ds = p (do.v - delta), dq = scale ds k, dk = scale ds^T q,
        dv = p^T do, dbias = sum of ds over the pairs of a bucket
  bias  attn with the bias: bucket b holds the distances from starts[b] up to
        starts[b + 1] - 1; the first half of the buckets one distance each, the
        rest in equal ratios up to max_distance
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


# ---- the cases -------------------------------------------------------------------

def _qk(name, direction, tokens, heads, kv_heads, dim, dtype, weights="same", rot=None, interleaved=False, seqs=1):
    """weights: type of the norms' weights and of their gradients ("same" as
    the activations, or "f32"); seqs: sequences the tokens are split into."""
    return dict(name=name, op="qk", dir=direction, tokens=tokens, seqs=seqs, ragged=seqs > 1, heads=heads,
                kv_heads=kv_heads, dim=dim, dtype=dtype, weights=weights, rot=dim if rot is None else rot,
                interleaved=interleaved)


def _attn(name, direction, tokens, seqs, ragged, heads, kv_heads, dim, dtype, window=0, sinks=0, buckets=0,
          max_distance=0, weights="same"):
    return dict(name=name, op="bias" if buckets else "attn", dir=direction, tokens=tokens, seqs=seqs, ragged=ragged,
                heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, window=window, sinks=sinks, buckets=buckets,
                max_distance=max_distance, weights=weights)


def listed():
    return [
        # one token's queries and keys, hidden 1600: bound by the launch
        _qk("qk_fwd_token", "fwd", 1, 25, 25, 64, "f16"),
        # 8 sequences of 1024 positions, hidden 1600
        _qk("qk_fwd_h1600", "fwd", 8192, 25, 25, 64, "f16"),
        # their backward pass with the gradients of both norms' weights
        _qk("qk_bwd_h1600", "bwd", 8192, 25, 25, 64, "f16"),
        # hidden 8192 with shared key heads, packed sequences, fp32 weights
        _qk("qk_bwd_h8192", "bwd", 16384, 64, 8, 128, "bf16", weights="f32", interleaved=True, seqs=7),
        # two short packed sequences: latency
        _attn("attn_fwd_small", "fwd", 131, 2, True, 25, 25, 64, "f16", window=64, sinks=4),
        # a GPT-2 block's attention: 8 sequences of 1024 positions, every earlier one visible
        _attn("attn_fwd_h1600", "fwd", 8192, 8, False, 25, 25, 64, "f16"),
        # hidden 8192, shared key heads, a window and four first tokens
        _attn("attn_fwd_h8192", "fwd", 8192, 2, False, 64, 8, 128, "bf16", window=512, sinks=4),
        # the backward pass in a GPT-2 block
        _attn("attn_bwd_h1600", "bwd", 8192, 8, False, 25, 25, 64, "f16"),
        # packed sequences of odd lengths at hidden 8192: the largest
        _attn("attn_bwd_h8192", "bwd", 8191, 3, True, 64, 8, 128, "bf16", window=1024, sinks=16),
        # a GPT-2 block with a learned bias in place of learned positions
        _attn("bias_fwd_h1600", "fwd", 8192, 8, False, 25, 25, 64, "f16", buckets=32, max_distance=128),
        # its backward pass with the bias' gradient
        _attn("bias_bwd_h1600", "bwd", 8192, 8, False, 25, 25, 64, "f16", buckets=32, max_distance=128),
        # odd lengths and a head size between the powers of two, a window beside the bias, fp32 bias
        _attn("bias_bwd_odd", "bwd", 4099, 5, True, 12, 3, 80, "bf16", window=700, sinks=1, buckets=24,
              max_distance=500, weights="f32"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op, direction = rng.choice(["qk", "attn", "attn", "bias", "bias"]), rng.choice(["fwd", "bwd"])
    kv = rng.choice([1, 2, 3, 4, 5, 8, 16, 25])
    heads = kv * rng.choice([1, 1, 2, 4, 8])
    weights = rng.choice(["same", "f32"])
    dim = rng.choice([64, 64, 128, 128, 8 * rng.randint(1, 16)])
    if op == "qk":
        dtype = rng.choice(["f16", "bf16", "f32"])
        tokens = _log(rng, 1, min(1 << 16, (1 << 27) // (heads * dim)))
        rot = dim if rng.random() < 0.7 else 2 * rng.randint(0, dim // 2)
        case = _qk(None, direction, tokens, heads, kv, dim, dtype, weights, rot, rng.random() < 0.5,
                   min(tokens, rng.choice([1, 1, 2, 5, 9])))
        del case["name"]
        return case
    dtype = rng.choice(["f16", "bf16"])
    longest = max(2.0, math.sqrt(2.0 ** 30 / heads))              # pairs of the padded score matrices
    seqs = rng.choice([1, 1, 2, 3, 4, 7])
    ragged = seqs > 1 and rng.random() < 0.7
    # a query that sees only itself has gradients of 0, of which the roundings alone would be compared
    least = 1 if direction == "fwd" else 2
    tokens = seqs * max(least, _log(rng, 1, longest / math.sqrt(seqs)) * (2 if ragged else 3) // 3)
    if ragged:
        tokens += rng.randint(0, 2)
    window = rng.choice([0, 0, least, _log(rng, 2, 4096)])
    sinks = rng.choice([0, 1, 4, rng.randint(1, 200)]) if window else 0
    buckets = 2 * rng.randint(1, 32) if op == "bias" else 0
    case = _attn(None, direction, tokens, seqs, ragged, heads, kv, dim, dtype, window, sinks, buckets,
                 buckets // 2 + _log(rng, 1, 2000) if buckets else 0, weights)
    del case["name"]
    return case


def _lengths(case):
    """The sequences' lengths: equal, or parts of the tokens that go by the case's own numbers."""
    n, t = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [t // n] * n
    r = random.Random(t * 1000 + n)
    parts = [0.5 + r.random() for _ in range(n)]
    ends = [int(round(t * sum(parts[:i + 1]) / sum(parts))) for i in range(n)]
    return [b - a for a, b in zip([0] + ends, ends)]


def _starts(case):
    """The first distance of each bucket: the border of b + half, half * (max_distance / half)^(b / half), rounded up
    (a whole number stays: it is looked for in whole numbers)."""
    n, most = case["buckets"], case["max_distance"]
    half = n // 2
    out = list(range(half))
    for b in range(n - half):
        d = max(half, int(half * (most / half) ** (b / (n - half))) - 2)
        while d ** (n - half) * half ** b < most ** b * half ** (n - half):
            d += 1
        out.append(max(d, out[-1] + 1) if out else d)
    return out


def _pairs(case):
    """Visible (query, key) pairs over all the sequences."""
    total = 0
    for n in _lengths(case):
        i = np.arange(n, dtype=np.int64)
        w = case["window"]
        total += int(np.minimum(i + 1, w).sum() + np.minimum(case["sinks"], np.maximum(0, i - w + 1)).sum()) if w else \
            n * (n + 1) // 2
    return total


def work(case):
    """Each input read once and each output written once; two operations for each product."""
    n, size, t, d = case["tokens"], SIZE[case["dtype"]], case["tokens"], case["dim"]
    hq, hk, fwd = case["heads"], case["kv_heads"], case["dir"] == "fwd"
    wsize = size if case["weights"] == "same" else 4
    if case["op"] == "qk":
        e = n * (hq + hk) * d
        return {"bytes": (2 if fwd else 3) * e * size + (2 if fwd else 4) * d * wsize + min(t, max(_lengths(case))) * case["rot"] * 4
                + 4 * t, "flops": (9 if fwd else 17) * e}
    pairs = _pairs(case)
    table = hq * case["buckets"] * wsize
    if fwd:
        return {"bytes": t * d * size * 2 * (hq + hk) + 4 * t * hq + table, "flops": 4 * d * pairs * hq}
    return {"bytes": t * d * size * 4 * (hq + hk) + 4 * t * hq + 2 * table, "flops": 10 * d * pairs * hq}


# ---- inputs ------------------------------------------------------------------------

def _heads(case, g, heads, scale, spread=0.0):
    """(tokens, heads, dim) values of the case's type: normal, with a part that
    all tokens of a head share."""
    t = torch.randn(case["tokens"], heads, case["dim"], generator=g, device="cuda")
    t = (t + spread * torch.randn(1, heads, case["dim"], generator=g, device="cuda")) * scale
    return t.to(TYPES[case["dtype"]])


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & ((1 << 62) - 1))
    lengths = _lengths(case)
    W = TYPES[case["dtype"] if case["weights"] == "same" else "f32"]
    s = {"case": case, "bias": None,
         "offsets": torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")}
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "qk":
        s["q"], s["k"] = _heads(case, g, hq, 1.5, 0.7), _heads(case, g, hk, 1.5, 0.7)
        s["wq"], s["wk"] = ((1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(W) for _ in range(2))
        longest, half = max(lengths), case["rot"] // 2
        angle = torch.arange(longest, dtype=torch.float64, device="cuda")[:, None] * torch.pow(
            torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
            torch.arange(half, dtype=torch.float64, device="cuda") * (-1.0 / max(half, 1)))
        s["table"] = torch.stack([angle.cos(), angle.sin()], 2).float()
        start = torch.repeat_interleave(s["offsets"][:-1].long(), torch.tensor(lengths, device="cuda"))
        s["positions"] = (torch.arange(case["tokens"], device="cuda") - start).int()
        if case["dir"] == "bwd":
            s["dq"], s["dk"] = _heads(case, g, hq, 0.05), _heads(case, g, hk, 0.05)
        return s
    s["scale"] = d ** -0.5
    s["q"], s["k"], s["v"] = _heads(case, g, hq, 1.0, 0.5), _heads(case, g, hk, 1.0, 0.5), _heads(case, g, hk, 1.0, 0.3)
    if case["buckets"]:
        s["starts"] = _starts(case)
        s["bias"] = (0.5 * torch.randn(hq, case["buckets"], generator=g, device="cuda")).to(W)
    if case["dir"] == "bwd":
        s["do"] = _heads(case, g, hq, 0.05)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(hq, case["tokens"], device="cuda")
        for a, b in zip(s["offsets"][:-1].tolist(), s["offsets"][1:].tolist()):
            for h in range(hq):
                p = _scores64(s, a, b, h)
                lse = torch.logsumexp(p, 1)
                s["lse"][h, a:b] = lse.float()
                s["o"][a:b, h] = (torch.exp(p - lse[:, None]).float() @ s["v"][a:b, h * hk // hq].float()).to(s["o"].dtype)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import zero_partitioned_mixed_flatten_amd as Z
        if case["op"] == "qk":
            s["out"] = [torch.empty_like(s["q"]), torch.empty_like(s["k"])]
            if case["dir"] == "bwd":
                s["out"] += [torch.empty_like(s["wq"]), torch.empty_like(s["wk"])]
                s["ws"] = torch.empty(max(16, Z.zero_qk_workspace_bytes(case["tokens"], case["heads"], case["kv_heads"], case["dim"])),
                                      dtype=torch.uint8, device="cuda")
        else:
            s["params"] = Z.attention_params(case["heads"], case["kv_heads"], case["dim"], window=case["window"],
                                             sinks=case["sinks"], starts=s.get("starts"))
            if case["dir"] == "fwd":
                s["out"] = [torch.empty_like(s["q"]), torch.empty(case["heads"], case["tokens"], device="cuda")]
            else:
                s["out"] = [torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"]),
                            torch.empty_like(s["bias"]) if case["buckets"] else None]
                s["ws"] = torch.empty(max(16, Z.zero_attention_workspace_bytes(s["params"], case["tokens"], case["seqs"])),
                                      dtype=torch.uint8, device="cuda")
    return s


# ---- the calls -----------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import zero_partitioned_mixed_flatten_amd as Z
    c, out = s["case"], s["out"]
    if c["op"] == "qk":
        if c["dir"] == "fwd":
            Z.zero_qk_norm_rope_fwd(out[0], out[1], s["q"], s["k"], s["wq"], s["wk"], s["table"], EPS,
                                    positions=s["positions"], interleaved=c["interleaved"])
            return {"q": out[0], "k": out[1]}
        Z.zero_qk_norm_rope_bwd(out[0], out[1], out[2], out[3], s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"],
                                s["table"], EPS, positions=s["positions"], interleaved=c["interleaved"],
                                workspace=s["ws"])
        return {"dq": out[0], "dk": out[1], "dwq": out[2], "dwk": out[3]}
    where = {"offsets": s["offsets"]} if c["ragged"] else {"sequences": c["seqs"]}
    if c["dir"] == "fwd":
        Z.zero_attention_fwd(out[0], out[1], s["q"], s["k"], s["v"], s["params"], bias=s["bias"], **where)
        return {"o": out[0], "lse": out[1]}
    Z.zero_attention_bwd(out[0], out[1], out[2], out[3], s["do"], s["o"], s["lse"], s["q"], s["k"], s["v"], s["params"],
                         bias=s["bias"], workspace=s["ws"], **where)
    return {"dq": out[0], "dk": out[1], "dv": out[2], **({"dbias": out[3]} if c["buckets"] else {})}


# ---- the plain form ---------------------------------------------------------------------

def _turn(u, table, positions, rot, interleaved, back):
    """The first `rot` elements of u (tokens, heads, dim) turned by their positions."""
    t = table[positions.long()][:, None]
    c, s = t[..., 0], -t[..., 1] if back else t[..., 1]
    r = u[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    x, y = a * c - b * s, b * c + a * s
    r = torch.stack([x, y], -1).flatten(-2) if interleaved else torch.cat([x, y], -1)
    return torch.cat([r, u[..., rot:]], -1)


def _qk_plain(s, x, w, dy):
    c = s["case"]
    x, w = x.float(), w.float()
    turn = (s["table"], s["positions"], c["rot"], c["interleaved"])
    rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    h = x * rstd
    if dy is None:
        return _turn(h * w, *turn, False)
    g = _turn(dy.float(), *turn, True)
    dw = (g * h).sum((0, 1))
    g = g * w
    return rstd * (g - h * (g * h).mean(-1, keepdim=True)), dw


def _run_plain(s):
    c = s["case"]
    T = TYPES[c["dtype"]]
    W = TYPES[c["dtype"] if c["weights"] == "same" else "f32"]
    if c["op"] == "qk":
        if c["dir"] == "fwd":
            return {"q": _qk_plain(s, s["q"], s["wq"], None).to(T), "k": _qk_plain(s, s["k"], s["wk"], None).to(T)}
        (dq, dwq), (dk, dwk) = _qk_plain(s, s["q"], s["wq"], s["dq"]), _qk_plain(s, s["k"], s["wk"], s["dk"])
        return {"dq": dq.to(T), "dk": dk.to(T), "dwq": dwq.to(W), "dwk": dwk.to(W)}

    # sequences side by side, padded to the longest: (sequences, kv_heads, group, length, dim)
    n, hq, hk, d = c["seqs"], c["heads"], c["kv_heads"], c["dim"]
    first, length = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    longest = max(_lengths(c))
    at = torch.arange(longest, device="cuda")
    inside = at[None] < length[:, None]
    index = torch.where(inside, first[:, None] + at[None], 0)
    spread = lambda t: t[index].float().masked_fill_(~inside[:, :, None, None], 0.0).view(
        n, longest, hk, -1, d).permute(0, 2, 3, 1, 4).contiguous()
    packed = lambda t: t.permute(0, 3, 1, 2, 4).reshape(n, longest, -1, d)[inside]
    q, k, v = spread(s["q"]), spread(s["k"]), spread(s["v"])
    far = at[:, None] - at[None]
    seen = far >= 0
    if c["window"]:
        seen = seen & ((far < c["window"]) | (at[None] < c["sinks"]))
    p = torch.matmul(q * s["scale"], k.transpose(-1, -2).contiguous())
    if c["buckets"]:
        bucket = torch.bucketize(far.clamp(min=0), torch.tensor(s["starts"], device="cuda"), right=True) - 1
        p += s["bias"].float()[:, bucket].view(hk, hq // hk, longest, longest)
    p = p.masked_fill_(~seen, -math.inf)
    if c["dir"] == "fwd":
        m = p.amax(-1, keepdim=True)
        p = torch.exp(p - m)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, v) / total
        lse = (m + torch.log(total)).reshape(n, hq, longest).permute(0, 2, 1)[inside]
        return {"o": packed(o).to(T), "lse": lse.t().contiguous()}
    rows = lambda t: t[index].masked_fill_(~inside[:, :, None], 0.0).view(n, longest, hk, -1).permute(0, 2, 3, 1)[..., None]
    do = spread(s["do"])
    delta = rows((s["do"].float() * s["o"].float()).sum(-1))
    p = torch.exp(p - rows(s["lse"].t()))
    p = p.masked_fill_(~inside[:, None, None, :, None], 0.0)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    ds = p * (torch.matmul(do, v.transpose(-1, -2).contiguous()) - delta)
    out = {"dq": packed(torch.matmul(ds, k) * s["scale"]).to(T),
           "dk": packed((torch.matmul(ds.transpose(-1, -2), q) * s["scale"]).sum(2, keepdim=True)).to(T),
           "dv": packed(dv).to(T)}
    if c["buckets"]:
        ds = ds.sum(0).view(hq, longest * longest)
        out["dbias"] = torch.zeros(hq, c["buckets"], device="cuda").index_add_(1, bucket.flatten(), ds).to(W)
    return out


# ---- the definition in 64 bits ------------------------------------------------------------

def _scores64(s, a, b, h):
    """Head h's scores of the sequence in tokens [a, b), -inf where not visible."""
    c = s["case"]
    i = torch.arange(b - a, device="cuda")
    dist = i.view(-1, 1) - i.view(1, -1)
    p = (s["q"][a:b, h].double() @ s["k"][a:b, h * c["kv_heads"] // c["heads"]].double().T.contiguous()) * s["scale"]
    if c["buckets"]:
        which = torch.zeros_like(dist)
        for first in s["starts"][1:]:
            which += dist >= first
        p += s["bias"][h].double()[which]
    hidden = dist < 0
    if c["window"]:
        hidden |= (dist >= c["window"]) & (i.view(1, -1) >= c["sinks"])
    return p.masked_fill(hidden, -math.inf)


def _qk_exact(s, x, w, dy):
    c = s["case"]
    x, w, rot, d = x.double(), w.double(), c["rot"], c["dim"]
    t = s["table"].double()[s["positions"].long()].view(-1, 1, rot // 2, 2)
    first = torch.arange(rot // 2, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else rot // 2)

    def turned(u, sign):
        out = u.clone()
        out[:, :, first] = u[:, :, first] * t[..., 0] - sign * u[:, :, second] * t[..., 1]
        out[:, :, second] = u[:, :, second] * t[..., 0] + sign * u[:, :, first] * t[..., 1]
        return out

    rstd = (x.pow(2).sum(2, keepdim=True) / d + EPS).pow(-0.5)
    if dy is None:
        return turned(x * rstd * w, 1.0)
    g = turned(dy.double(), -1.0)
    dw = (g * x * rstd).sum(0).sum(0)
    g = g * w
    return rstd * g - x * rstd.pow(3) * (g * x).sum(2, keepdim=True) / d, dw


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "qk":
        if case["dir"] == "fwd":
            return {"q": _qk_exact(s, s["q"], s["wq"], None), "k": _qk_exact(s, s["k"], s["wk"], None)}
        (dq, dwq), (dk, dwk) = _qk_exact(s, s["q"], s["wq"], s["dq"]), _qk_exact(s, s["k"], s["wk"], s["dk"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    hq, hk, t, d = case["heads"], case["kv_heads"], case["tokens"], case["dim"]
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")
    fwd = case["dir"] == "fwd"
    out = {"o": new(t, hq, d), "lse": new(hq, t)} if fwd else {"dq": new(t, hq, d), "dk": new(t, hk, d), "dv": new(t, hk, d)}
    if not fwd and case["buckets"]:
        out["dbias"] = new(hq, case["buckets"])
    edges = s["offsets"].tolist()
    for a, b in zip(edges, edges[1:]):
        if a == b:
            continue
        dist = torch.arange(b - a, device="cuda")
        dist = dist.view(-1, 1) - dist.view(1, -1)
        for h in range(hq):
            p, g = _scores64(s, a, b, h), h * hk // hq
            if fwd:
                lse = torch.logsumexp(p, 1)
                out["o"][a:b, h] = torch.exp(p - lse[:, None]) @ s["v"][a:b, g].double()
                out["lse"][h, a:b] = lse
                continue
            p = torch.exp(p - s["lse"][h, a:b].double()[:, None])
            do = s["do"][a:b, h].double()
            ds = do @ s["v"][a:b, g].double().T.contiguous()
            ds -= (do * s["o"][a:b, h].double()).sum(1, keepdim=True)
            ds *= p
            out["dq"][a:b, h] = s["scale"] * (ds @ s["k"][a:b, g].double())
            out["dk"][a:b, g] += s["scale"] * (ds.T @ s["q"][a:b, h].double())
            out["dv"][a:b, g] += p.T @ do
            for i in range(case["buckets"]):
                low = s["starts"][i]
                high = s["starts"][i + 1] if i + 1 < case["buckets"] else 1 << 40
                # the diagonals low <= i - j < high: what lies on or below the one, less what lies on or below the other
                part = torch.tril(ds, -low) - (torch.tril(ds, -high) if high < b - a else 0.0)
                out["dbias"][h, i] += part.sum()
    return out
