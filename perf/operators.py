"""Measured cases of the layer operators around a transformer block's residual
stream: dropout whose mask is recomputed from a counter-based generator, layer
norm with the gradients of its weights, and the two joined (bias + dropout +
residual + layer norm), forward and backward.

`run` computes a case either in plain torch operations (own = False) or with
the framework's entry points (own = True).

The arithmetic, for a rows x cols matrix of element type T (everything in
32 bits, rounded to T once where it is stored):

  generator  Philox4x32-10 (Salmon et al. 2011); key = the 64-bit seed,
             counter = (g low, g high, site, step) with
             g = row * ceil(cols / 8) + col // 8; element col takes the
             16-bit word col % 8 of the four outputs and is dropped when it
             is below t = floor(65536 p + 1/2)
  D(v)       = kept ? v * 65536 / (65536 - t) : 0
  dropout    out = residual + D(x + bias); dx = D(dout), dbias = sum of dx
  layer norm y = (x - mean) * rstd * w + b, rstd = 1 / sqrt(var + eps);
             h = (x - mean) * rstd, g = dy * w,
             dx = rstd * (g - mean(g) - h * mean(g h)) + dres,
             dw = sum of dy * h, db = sum of dy over the rows
  joined     r = residual + D(x + bias), stored in T, then the layer norm of
             the stored r; backward: dr = the layer norm's dx at r,
             dx = D(dr), dbias = sum of dx
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


# ---- the cases -------------------------------------------------------------------

def _case(name, op, direction, rows, cols, dtype, weights="same", p=0.1, pad=0, extra=True):
    """weights: type of w, b, bias and of their gradients ("same" as the
    matrices, or "f32"); pad: elements between the rows; extra: with the
    optional inputs (bias and residual, or the residual stream's gradient)."""
    return dict(name=name, op=op, dir=direction, rows=rows, cols=cols, dtype=dtype, weights=weights, p=p, pad=pad,
                extra=extra)


def listed():
    return [
        # one token's final norm, hidden 1600: bound by the launch
        _case("norm_fwd_token", "layernorm", "fwd", 1, 1600, "f16"),
        # 8 sequences of 1024 positions, hidden 1600: a GPT-2 block's norm
        _case("norm_fwd_h1600", "layernorm", "fwd", 8192, 1600, "f16", extra=False),
        # its backward pass, with the gradient of the residual stream added
        _case("norm_bwd_h1600", "layernorm", "bwd", 8192, 1600, "f16"),
        # odd width, padded rows, fp32 throughout
        _case("norm_bwd_odd_f32", "layernorm", "bwd", 4099, 1601, "f32", pad=3, extra=False),
        # attention probabilities of one layer: 25 heads, 1024 x 1024
        _case("drop_fwd_probs", "dropout", "fwd", 25600, 1024, "f16", extra=False),
        # bias + dropout + residual after a hidden-8192 projection
        _case("drop_fwd_h8192", "dropout", "fwd", 16384, 8192, "bf16", weights="f32"),
        # a short micro-batch's backward with its bias gradient: latency
        _case("drop_bwd_small", "dropout", "bwd", 96, 1600, "bf16"),
        # the joined forward in a GPT-2 block
        _case("join_fwd_h1600", "dropout_layernorm", "fwd", 8192, 1600, "f16"),
        # two ragged sequences: joined forward at a wide block's hidden size
        _case("join_fwd_h8192", "dropout_layernorm", "fwd", 1531, 8192, "bf16", weights="f32"),
        # a short micro-batch's joined backward: latency and the short fold
        _case("join_bwd_small", "dropout_layernorm", "bwd", 128, 1600, "f16"),
        # the joined backward in a GPT-2 block
        _case("join_bwd_h1600", "dropout_layernorm", "bwd", 8192, 1600, "f16"),
        # the joined backward at hidden 8192, fp32 weight gradients: the largest
        _case("join_bwd_h8192", "dropout_layernorm", "bwd", 16384, 8192, "bf16", weights="f32"),
    ]


def draw(rng):
    dtype = rng.choice(["f16", "bf16", "f32"])
    most = (1 << 27) * 2 // SIZE[dtype]                         # elements of the largest listed case
    cols = int(round(math.exp(rng.uniform(0.0, math.log(20000.0)))))
    if rng.random() < 0.5:
        cols = max(8, cols // 8 * 8)
    rows = int(round(math.exp(rng.uniform(0.0, math.log(min(1 << 18, most // cols))))))
    return dict(op=rng.choice(["dropout", "layernorm", "dropout_layernorm"]), dir=rng.choice(["fwd", "bwd"]),
                rows=rows, cols=cols, dtype=dtype, weights=rng.choice(["same", "f32"]),
                p=rng.choice([0.0, 0.05, 0.1, 0.2, 0.5, round(rng.uniform(0.01, 0.9), 3)]),
                pad=rng.choice([0, 0, 0, 1, 8, 24]), extra=rng.random() < 0.7)


def work(case):
    """Each input read once and each output written once."""
    e, n = case["rows"] * case["cols"], SIZE[case["dtype"]]
    wsize = n if case["weights"] == "same" else 4
    join, norm, fwd = case["op"] == "dropout_layernorm", case["op"] != "dropout", case["dir"] == "fwd"
    if fwd:
        arrays = 4 if join else (3 if case["op"] == "dropout" and case["extra"] else 2)
        if join and not case["extra"]:
            arrays = 3
        vectors = (2 if norm else 0) + (1 if case["extra"] and not (norm and not join) else 0)
    else:
        arrays = {"dropout": 2, "layernorm": 3, "dropout_layernorm": 4}[case["op"]]
        if norm and case["extra"]:
            arrays += 1
        vectors = {"dropout": 1, "layernorm": 3, "dropout_layernorm": 4}[case["op"]]
    total = arrays * e * n + vectors * case["cols"] * wsize + (8 * case["rows"] if norm else 0)
    per = {("dropout", True): 3, ("dropout", False): 2, ("layernorm", True): 8, ("layernorm", False): 14,
           ("dropout_layernorm", True): 11, ("dropout_layernorm", False): 17}[(case["op"], fwd)]
    return {"bytes": total, "flops": per * e}


# ---- inputs ------------------------------------------------------------------------

def _matrix(case, g, scale, offset=False):
    """rows x cols values of the case's type, rows `pad` elements apart:
    normal, some columns much larger (as a residual stream has them), an
    offset for each column."""
    rows, cols = case["rows"], case["cols"]
    t = torch.empty(rows, cols + case["pad"], dtype=TYPES[case["dtype"]], device="cuda")
    m = t[:, :cols]
    big = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 8.0, 1.0) * scale
    off = torch.randn(cols, generator=g, device="cuda") * (0.3 * scale if offset else 0.0)
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        k = min(step, rows - r)
        v = torch.randn(k, cols, generator=g, device="cuda")
        m[r:r + k] = (v * big + off).to(m.dtype)
    return m


def _vector(case, g, around, scale):
    dtype = TYPES[case["dtype"] if case["weights"] == "same" else "f32"]
    return (around + scale * torch.randn(case["cols"], generator=g, device="cuda")).to(dtype)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & ((1 << 62) - 1))
    norm, drop = case["op"] != "dropout", case["op"] != "layernorm"
    s = {"case": case, "residual": None, "bias": None, "dres": None,
         "seed": (int(seed) * 0x9E3779B97F4A7C15 + 12345) & ((1 << 63) - 1), "step": 2, "site": 7}
    if norm:
        s["w"] = _vector(case, g, 1.0, 0.1)
    if case["dir"] == "fwd":
        s["x"] = _matrix(case, g, 1.0, True)
        if norm:
            s["b"] = _vector(case, g, 0.0, 0.1)
        if drop and case["extra"]:
            s["residual"] = _matrix(case, g, 2.0, True)
            s["bias"] = _vector(case, g, 0.0, 0.1)
        return s
    s["dy"] = _matrix(case, g, 0.05)
    if norm:
        s["x"] = _matrix(case, g, 2.0, True)
        rows, step = case["rows"], max(1, (1 << 26) // case["cols"])
        s["mean"] = torch.empty(rows, device="cuda")
        s["rstd"] = torch.empty(rows, device="cuda")
        for r in range(0, rows, step):
            v = s["x"][r:r + step].double()
            s["mean"][r:r + step] = v.mean(1).float()
            s["rstd"][r:r + step] = (v.var(1, unbiased=False) + EPS).rsqrt().float()
        if case["extra"]:
            s["dres"] = _matrix(case, g, 0.05)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    rows, cols = case["rows"], case["cols"]
    like = lambda: torch.empty(rows, cols + case["pad"], dtype=TYPES[case["dtype"]], device="cuda")[:, :cols]
    vec = lambda: torch.empty(cols, dtype=TYPES[case["dtype"] if case["weights"] == "same" else "f32"], device="cuda")
    if not own:
        return s
    import zero_partitioned_mixed_flatten_amd as Z
    if case["op"] != "layernorm":
        s["rng"] = torch.zeros(Z.RNG_BYTES, dtype=torch.uint8, device="cuda")
        Z.zero_rng_init(s["rng"], s["seed"])
        for _ in range(s["step"]):
            Z.zero_rng_advance(s["rng"])
    if case["dir"] == "fwd":
        s["o_y"] = like()
        if case["op"] == "dropout_layernorm":
            s["o_r"] = like()
        if case["op"] != "dropout":
            s["o_mean"] = torch.empty(rows, device="cuda")
            s["o_rstd"] = torch.empty(rows, device="cuda")
    else:
        s["o_dx"] = like()
        if case["op"] == "dropout_layernorm":
            s["o_dr"] = like()
        if case["op"] != "dropout":
            s["o_dw"], s["o_db"] = vec(), vec()
        if case["op"] != "layernorm":
            s["o_dbias"] = vec()
        s["ws"] = torch.empty(max(16, Z.zero_layer_workspace_bytes(rows, cols)), dtype=torch.uint8, device="cuda")
    return s


# ---- the calls -----------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import zero_partitioned_mixed_flatten_amd as Z
    c = s["case"]
    op, fwd = c["op"], c["dir"] == "fwd"
    if op == "dropout" and fwd:
        Z.zero_dropout_fwd(s["o_y"], s["x"], c["p"], s["rng"], s["site"], residual=s["residual"], bias=s["bias"])
        return {"out": s["o_y"]}
    if op == "dropout":
        Z.zero_dropout_bwd(s["o_dx"], s["dy"], c["p"], s["rng"], s["site"], dbias=s["o_dbias"], workspace=s["ws"])
        return {"dx": s["o_dx"], "dbias": s["o_dbias"]}
    if op == "layernorm" and fwd:
        Z.zero_layernorm_fwd(s["o_y"], s["o_mean"], s["o_rstd"], s["x"], s["w"], s["b"], EPS)
        return {"y": s["o_y"], "mean": s["o_mean"], "rstd": s["o_rstd"]}
    if op == "layernorm":
        Z.zero_layernorm_bwd(s["o_dx"], s["o_dw"], s["o_db"], s["dy"], s["x"], s["mean"], s["rstd"], s["w"],
                             dres=s["dres"], workspace=s["ws"])
        return {"dx": s["o_dx"], "dw": s["o_dw"], "db": s["o_db"]}
    if fwd:
        Z.zero_dropout_layernorm_fwd(s["o_r"], s["o_y"], s["o_mean"], s["o_rstd"], s["x"], s["residual"], s["bias"],
                                     s["w"], s["b"], EPS, c["p"], s["rng"], s["site"])
        return {"r": s["o_r"], "y": s["o_y"], "mean": s["o_mean"], "rstd": s["o_rstd"]}
    Z.zero_dropout_layernorm_bwd(s["o_dx"], s["o_dr"], s["o_dw"], s["o_db"], s["o_dbias"], s["dy"], s["dres"], s["x"],
                                 s["mean"], s["rstd"], s["w"], c["p"], s["rng"], s["site"], workspace=s["ws"])
    return {"dx": s["o_dx"], "dr": s["o_dr"], "dw": s["o_dw"], "db": s["o_db"], "dbias": s["o_dbias"]}


# ---- the plain form ---------------------------------------------------------------------

def _keep(s):
    """The kept elements (rows x cols truth values) and the factor."""
    c = s["case"]
    t = int(math.floor(c["p"] * 65536.0 + 0.5))
    if t == 0:
        return None, 1.0
    gpr = -(-c["cols"] // 8)
    m = 0xFFFFFFFF
    g = torch.arange(c["rows"] * gpr, dtype=torch.int64, device="cuda")
    c0, c1 = g & m, g >> 32
    c2, c3 = torch.full_like(g, s["site"]), torch.full_like(g, s["step"])
    k0, k1 = s["seed"] & m, s["seed"] >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57               # low 64 bits of the products, as int64
        c0, c1, c2, c3 = ((b >> 32) & m) ^ c1 ^ k0, b & m, ((a >> 32) & m) ^ c3 ^ k1, a & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    halves = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 1)
    keep = (halves >= t).reshape(c["rows"], gpr * 8)[:, :c["cols"]]
    return keep, (65536.0 / (65536 - t) if t < 65536 else 0.0)


def _dropped(v, keep, factor):
    return v if keep is None else torch.where(keep, v * torch.tensor(factor, dtype=v.dtype, device=v.device), 0.0)


def _run_plain(s):
    c = s["case"]
    T = TYPES[c["dtype"]]
    W = TYPES[c["dtype"] if c["weights"] == "same" else "f32"]
    op, norm, drop = c["op"], c["op"] != "dropout", c["op"] != "layernorm"
    keep, factor = _keep(s) if drop else (None, 1.0)
    if c["dir"] == "fwd":
        v = s["x"].float()
        out = {}
        if drop:
            if s["bias"] is not None:
                v = v + s["bias"].float()
            v = _dropped(v, keep, factor)
            if s["residual"] is not None:
                v = s["residual"].float() + v
            out["out" if op == "dropout" else "r"] = v.to(T)
            v = v.to(T).float()
        if norm:
            mean = v.mean(1, keepdim=True)
            d = v - mean
            rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
            out["y"] = (d * rstd * s["w"].float() + s["b"].float()).to(T)
            out["mean"], out["rstd"] = mean.flatten(), rstd.flatten()
        return out
    e = s["dy"].float()
    out = {}
    if norm:
        rstd = s["rstd"][:, None]
        h = (s["x"].float() - s["mean"][:, None]) * rstd
        out["dw"], out["db"] = (e * h).sum(0).to(W), e.sum(0).to(W)
        g = e * s["w"].float()
        e = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        if s["dres"] is not None:
            e = e + s["dres"].float()
    if not drop:
        out["dx"] = e.to(T)
        return out
    if norm:
        out["dr"] = e.to(T)
    e = _dropped(e, keep, factor)
    out["dx"], out["dbias"] = e.to(T), e.sum(0).to(W)
    return out


# ---- the definition in 64 bits ------------------------------------------------------------

def _exact_factors(case, s):
    """rows x cols factors of D in 64 bits (0 where dropped), from products
    taken in 16-bit parts."""
    t = math.floor(case["p"] * 65536.0 + 0.5)
    rows, cols = case["rows"], case["cols"]
    if t <= 0:
        return torch.ones(1, 1, dtype=torch.float64, device="cuda")
    groups = (cols + 7) // 8
    index = torch.arange(rows, device="cuda")[:, None] * groups + torch.arange(groups, device="cuda")[None, :]

    def product(u, const):
        lo, hi = u & 0xFFFF, u >> 16
        p0, p1 = lo * const, hi * const                       # below 2^48 each
        low = (p0 & 0xFFFFFFFF) + ((p1 & 0xFFFF) << 16)
        return (p0 >> 32) + (p1 >> 16) + (low >> 32), low & 0xFFFFFFFF

    x = [index % (1 << 32), index // (1 << 32), torch.full_like(index, s["site"]), torch.full_like(index, s["step"])]
    key = [s["seed"] % (1 << 32), s["seed"] // (1 << 32)]
    for r in range(10):
        ka = (key[0] + r * 0x9E3779B9) % (1 << 32)
        kb = (key[1] + r * 0xBB67AE85) % (1 << 32)
        h0, l0 = product(x[0], 0xD2511F53)
        h1, l1 = product(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ ka, l1, h0 ^ x[3] ^ kb, l0]
    out = torch.empty(rows, groups, 8, dtype=torch.float64, device="cuda")
    for j in range(8):
        word = (x[j // 2] >> (16 * (j % 2))) % 65536
        out[:, :, j] = (word >= t).double() * (65536.0 / (65536 - t) if t < 65536 else 0.0)
    return out.reshape(rows, groups * 8)[:, :cols]


def exact(case, seed):
    s = _inputs(case, seed)
    n = case["cols"]
    join, norm = case["op"] == "dropout_layernorm", case["op"] != "dropout"
    if case["dir"] == "fwd":
        v, out = s["x"].double(), {}
        if case["op"] != "layernorm":
            if s["bias"] is not None:
                v += s["bias"].double()
            v *= _exact_factors(case, s)
            if s["residual"] is not None:
                v += s["residual"].double()
            out["r" if join else "out"] = v
        if norm:
            if join:                                          # the norm is of r as it is stored
                v = v.to(TYPES[case["dtype"]]).double()
            mean = v.sum(1) / n
            v = v - mean[:, None]
            rstd = (v.pow(2).sum(1) / n + EPS).pow(-0.5)
            out["y"] = v * rstd[:, None] * s["w"].double() + s["b"].double()
            out["mean"], out["rstd"] = mean, rstd
        return out
    dy, out = s["dy"].double(), {}
    if norm:
        h = (s["x"].double() - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        out["dw"], out["db"] = (dy * h).sum(0), dy.sum(0)
        g = dy * s["w"].double()
        c1, c2 = g.sum(1) / n, (g * h).sum(1) / n
        dy = (g - c1[:, None] - h * c2[:, None]) * s["rstd"].double()[:, None]
        if s["dres"] is not None:
            dy = dy + s["dres"].double()
        out["dr" if join else "dx"] = dy
        if not join:
            return out
    dy = dy * _exact_factors(case, s)
    out["dx"], out["dbias"] = dy, dy.sum(0)
    return out
