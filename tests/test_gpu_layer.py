"""The layer operators on the GPU against their 64-bit forms (layer_oracle.py):
every type, widths from one column to past what registers hold, odd widths,
padded and shifted rows, empty batches, rows whose mask leaves nothing,
infinities and NaN, other streams, captured graphs, offsets past 32 bits, and
the operators together with the shard step that consumes their gradients."""
import zlib

import numpy as np
import pytest
import torch

import layer_oracle as O

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402

KINDS = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
SHAPES = [(1, 1), (3, 1), (1, 8), (5, 3), (4, 64), (130, 65), (7, 129), (33, 513), (4, 1600), (131, 1600), (9, 1601),
          (1000, 24), (3, 4097), (5, 8192), (70, 5000), (2, 16391), (3, 33000), (600, 200)]


def log(*a):
    print("[layer]", *a, flush=True)


def gen(*words):
    g = torch.Generator()
    g.manual_seed(zlib.crc32(repr(words).encode()))
    return g


def matrix(g, rows, cols, kind, scale=1.0, offset=0.0, pad=0, shift=0):
    """rows x cols values on the GPU, rows `pad` elements apart, the first
    `shift` elements into its buffer; the buffer around them holds a canary."""
    buf = torch.full((shift + rows * (cols + pad) + 16,), 77.0, dtype=KINDS[kind])
    m = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_((torch.randn(rows, cols, generator=g) * scale + offset).to(KINDS[kind]))
    dev = buf.cuda()
    v = dev[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.buf, v.geometry = dev, (shift, rows, cols, pad)
    return v


def empty(rows, cols, kind, pad=0, shift=0):
    m = matrix(gen(0), rows, cols, kind, 0.0, 55.0, pad, shift)
    return m


def canary_ok(m):
    shift, rows, cols, pad = m.geometry
    b = m.buf.cpu().float()
    body = b[shift:shift + rows * (cols + pad)].view(rows, cols + pad)
    return bool((b[:shift] == 77).all() and (b[shift + rows * (cols + pad):] == 77).all() and (body[:, cols:] == 77).all())


def vector(g, cols, kind, around, scale, shift=0):
    t = torch.full((shift + cols + 8,), 33.0, dtype=KINDS[kind])
    t[shift:shift + cols] = (around + scale * torch.randn(cols, generator=g)).to(KINDS[kind])
    return t.cuda()[shift:shift + cols]


def f64(t):
    return t.detach().cpu().double().numpy()


def rng_state(seed, step):
    r = torch.zeros(Z.RNG_BYTES, dtype=torch.uint8, device="cuda")
    Z.zero_rng_init(r, seed)
    for _ in range(step):
        Z.zero_rng_advance(r)
    return r


def dirty_workspace(rows, cols):
    """A workspace full of NaN patterns: nothing in it may be read before it is written."""
    return torch.full((max(16, Z.zero_layer_workspace_bytes(rows, cols)),), 0xFF, dtype=torch.uint8, device="cuda")


def close(got, want, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = tuple(int(k[0]) for k in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first at {i}: got {got[i]!r}, want {want[i]!r}, "
                             f"bound {np.broadcast_to(bound, want.shape)[i]!r}")


def expect_r(x, residual, bias, kept, s):
    """residual + D(x + bias) in binary32, one rounding per operation, stored in
    the type: what the kernels must give bit for bit."""
    v = x.detach().cpu().float()
    if bias is not None:
        v = v + bias.detach().cpu().float()
    if kept is not None:
        v = torch.where(torch.from_numpy(kept), v * np.float32(s), torch.zeros(()))
    if residual is not None:
        v = residual.detach().cpu().float() + v
    return v.to(x.dtype)


def same_bits(got, want, what):
    g, w = got.detach().cpu().contiguous(), want.contiguous()
    v = torch.int32 if g.dtype == torch.float32 else torch.int16
    assert torch.equal(g.view(v), w.view(v)), (what, (g.float() - w.float()).abs().max())


def options(rows, cols, kind, op):
    """A spread of layouts and options over the shapes, by a hash of the case."""
    h = zlib.crc32(repr((rows, cols, kind, op)).encode())
    return dict(pad=(0, 3, 8)[h % 3], shift=(0, 1, 8)[h // 3 % 3], vec=(kind, "f32")[h // 9 % 2],
                extra=h // 18 % 3 != 0, p=(0.1, 0.5, 0.0, 0.9)[h // 54 % 4], accumulate=h // 216 % 2 == 1)


SEED = 0x1234567890ABCDEF


# ---- dropout -----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dropout(rows, cols, kind):
    o = options(rows, cols, kind, "dropout")
    log("dropout", rows, cols, kind, o)
    g = gen("dropout", rows, cols, kind)
    x = matrix(g, rows, cols, kind, pad=o["pad"], shift=o["shift"])
    res = matrix(g, rows, cols, kind, 2.0, pad=8 - o["pad"], shift=3) if o["extra"] else None
    bias = vector(g, cols, o["vec"], 0.0, 0.3, o["shift"]) if o["extra"] else None
    rng = rng_state(SEED, 2)
    out = empty(rows, cols, kind, pad=o["pad"], shift=1)
    Z.zero_dropout_fwd(out, x, o["p"], rng, 11, residual=res, bias=bias)
    kept, s = O.keep(rows, cols, o["p"], SEED, 2, 11), O.scale(o["p"])
    same_bits(out, expect_r(x, res, bias, kept, s), "out")
    assert canary_ok(out)
    # backward: the same mask, with and without the bias gradient
    dout = matrix(g, rows, cols, kind, 0.5, pad=o["pad"], shift=o["shift"])
    dx = empty(rows, cols, kind, pad=3, shift=o["shift"])
    Z.zero_dropout_bwd(dx, dout, o["p"], rng, 11)
    want = expect_r(dout, None, None, kept, s)
    same_bits(dx, want, "dx")
    dx2 = empty(rows, cols, kind, pad=o["pad"], shift=2)
    db = vector(g, cols, o["vec"], 1.0, 1.0, o["shift"])
    before = f64(db)
    Z.zero_dropout_bwd(dx2, dout, o["p"], rng, 11, dbias=db, accumulate=o["accumulate"],
                       workspace=dirty_workspace(rows, cols))
    same_bits(dx2, want, "dx with dbias")
    assert canary_ok(dx) and canary_ok(dx2)
    v = O.dropped(f64(dout), kept, s)
    sum_, e = O.column_sum(v, O.U * np.abs(v))
    if o["accumulate"]:
        sum_ = sum_ + before
        e = e + O.U * np.abs(sum_)
    close(db, sum_, O.stored(e, sum_, o["vec"]), "dbias")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("p", [0.0, 1.0, 1e-6, 0.99999, 2.0 ** -16, 0.25])
def test_dropout_probabilities(kind, p):
    """The ends of the range: nothing drawn, everything dropped, below and at
    the generator's resolution."""
    log("p", kind, p)
    g = gen("p", kind, p)
    x = matrix(g, 37, 203, kind)
    out = empty(37, 203, kind)
    Z.zero_dropout_fwd(out, x, p, rng_state(SEED, 0) if p else None, 1)
    same_bits(out, expect_r(x, None, None, O.keep(37, 203, p, SEED, 0, 1), O.scale(p)), p)


@pytest.mark.parametrize("kind", KINDS)
def test_dropped_infinities_and_nans_are_zero(kind):
    """What dropout removes leaves no trace, whatever it was; what it keeps
    comes through."""
    rows, cols = 24, 101
    kept = O.keep(rows, cols, 0.5, SEED, 1, 4)
    x = torch.ones(rows, cols)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")])
    x = torch.where(torch.from_numpy(kept), x, bad[torch.arange(rows * cols).view(rows, cols) % 3])
    x = x.to(KINDS[kind]).cuda()
    rng = rng_state(SEED, 1)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    db = torch.empty(cols, device="cuda")
    log("nan in dropped places", kind)
    Z.zero_dropout_fwd(out, x, 0.5, rng, 4)
    Z.zero_dropout_bwd(dx, x, 0.5, rng, 4, dbias=db, workspace=dirty_workspace(rows, cols))
    want = torch.from_numpy(kept).double() * 2.0
    assert torch.equal(out.cpu().double(), want) and torch.equal(dx.cpu().double(), want)
    assert torch.equal(db.cpu().double(), want.sum(0))
    # the joined form too: with a residual, the dropped places are the residual alone
    w, b = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    r, y = torch.empty_like(x), torch.empty_like(x)
    res = torch.full_like(x, 3.0)
    Z.zero_dropout_layernorm_fwd(r, y, None, None, x, res, None, w, b, EPS, 0.5, rng, 4)
    assert torch.equal(r.cpu().double(), want + 3.0)
    assert bool(torch.isfinite(y).all())
    # kept ones come through
    x2 = torch.where(torch.from_numpy(kept).cuda(), torch.full_like(x, float("inf")), torch.ones_like(x))
    Z.zero_dropout_fwd(out, x2, 0.5, rng, 4)
    assert torch.equal(torch.isinf(out).cpu(), torch.from_numpy(kept))


# ---- layer norm -----------------------------------------------------------------------------

def _check_fwd(x, y, mean, rstd, w, b, kind, eps=EPS):
    want, bound = O.norm_fwd(f64(x), 1.0 if w is None else f64(w)[None], 0.0 if b is None else f64(b)[None], eps, kind)
    close(mean, want[1], bound[1], "mean")
    close(rstd, want[2], bound[2], "rstd")
    close(y, want[0], bound[0], "y")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_layernorm_forward(rows, cols, kind):
    o = options(rows, cols, kind, "norm")
    log("layernorm fwd", rows, cols, kind, o)
    g = gen("norm", rows, cols, kind)
    x = matrix(g, rows, cols, kind, 1.5, 0.7, pad=o["pad"], shift=o["shift"])
    w = vector(g, cols, o["vec"], 1.0, 0.3, o["shift"])
    b = vector(g, cols, o["vec"], 0.0, 0.3, 1) if o["extra"] else None
    y = empty(rows, cols, kind, pad=8 - o["pad"], shift=o["shift"])
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    Z.zero_layernorm_fwd(y, mean, rstd, x, w, b, EPS)
    _check_fwd(x, y, mean, rstd, w, b, kind)
    assert canary_ok(y)
    y2 = empty(rows, cols, kind)
    Z.zero_layernorm_fwd(y2, None, None, x, w, b, EPS)              # the statistics are optional
    same_bits(y2, y.cpu(), "without statistics")
    Z.zero_layernorm_fwd(y2, None, None, x, None, None, EPS)        # and so are w and b
    _check_fwd(x, y2, mean, rstd, None, None, kind)


def _stats(x):
    v = x.double()
    return v.mean(1).float(), (v.var(1, unbiased=False) + EPS).rsqrt().float()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_layernorm_backward(rows, cols, kind):
    o = options(rows, cols, kind, "norm bwd")
    log("layernorm bwd", rows, cols, kind, o)
    g = gen("norm bwd", rows, cols, kind)
    x = matrix(g, rows, cols, kind, 1.5, 0.7, pad=o["pad"], shift=o["shift"])
    dy = matrix(g, rows, cols, kind, 0.5, pad=o["pad"], shift=1)
    dres = matrix(g, rows, cols, kind, 0.5, pad=3) if o["extra"] else None
    w = vector(g, cols, o["vec"], 1.0, 0.3, o["shift"])
    mean, rstd = _stats(x)
    dx = empty(rows, cols, kind, pad=8 - o["pad"], shift=o["shift"])
    dw, db = (vector(g, cols, "f32" if o["vec"] == kind else kind, 0.5, 1.0, 1) for _ in range(2))
    before = f64(dw), f64(db)
    Z.zero_layernorm_bwd(dx, dw, db, dy, x, mean, rstd, w, dres=dres, accumulate=o["accumulate"],
                         workspace=dirty_workspace(rows, cols))
    want, bound = O.norm_bwd(f64(dy), f64(x), f64(mean), f64(rstd), f64(w)[None], None if dres is None else f64(dres))
    close(dx, want[0], O.stored(bound[0], want[0], kind), "dx")
    assert canary_ok(dx)
    gk = "f32" if o["vec"] == kind else kind
    for name, got, i in (("dw", dw, 1), ("db", db, 2)):
        t, e = want[i], bound[i]
        if o["accumulate"]:
            t = t + before[i - 1]
            e = e + O.U * np.abs(t)
        close(got, t, O.stored(e, t, gk), name)
    # each gradient alone, and none: the same bits
    dw2, db2, dx2 = torch.zeros_like(dw), torch.zeros_like(db), empty(rows, cols, kind)
    Z.zero_layernorm_bwd(dx2, dw2, None, dy, x, mean, rstd, w, dres=dres, workspace=dirty_workspace(rows, cols))
    same_bits(dx2, dx.cpu(), "dx, dw only")
    Z.zero_layernorm_bwd(dx2, None, db2, dy, x, mean, rstd, w, dres=dres, workspace=dirty_workspace(rows, cols))
    if not o["accumulate"]:
        same_bits(dw2, dw.cpu(), "dw alone")
        same_bits(db2, db.cpu(), "db alone")
    Z.zero_layernorm_bwd(dx2, None, None, dy, x, mean, rstd, w, dres=dres)
    same_bits(dx2, dx.cpu(), "dx alone")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cols", [1, 7, 64, 1600, 8200, 20000])
def test_layernorm_special_rows(cols, kind):
    """Constant rows, rows of zeros, a row far from zero, a row with an inf and
    one with a NaN: each row depends on itself alone."""
    log("special rows", cols, kind)
    g = gen("special", cols, kind)
    x = torch.randn(9, cols, generator=g)
    x[1] = 0.0
    x[2] = 3.0
    x[3] = x[3] * 0.25 + 1000.0
    x[5, cols // 2] = float("inf")
    x[7, 0] = float("nan")
    x = x.to(KINDS[kind]).cuda()
    w, b = vector(g, cols, "f32", 1.0, 0.3), vector(g, cols, "f32", 0.5, 0.3)
    y, mean, rstd = torch.empty_like(x), torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    Z.zero_layernorm_fwd(y, mean, rstd, x, w, b, EPS)
    good = [0, 1, 2, 3, 4, 6, 8]
    _check_fwd(x[good], y[good], mean[good], rstd[good], w, b, kind)
    assert bool(torch.isnan(y[5]).all()) and bool(torch.isnan(y[7]).all())
    assert float(rstd[1]) == float(rstd[2]) == np.float32(1.0) / np.sqrt(np.float32(EPS))
    # backward: the broken rows' dx is NaN, every other row's is as without them
    dy = torch.randn(9, cols, generator=g).to(KINDS[kind]).cuda()
    dx, dx2 = torch.empty_like(x), torch.empty_like(x)
    Z.zero_layernorm_bwd(dx, None, None, dy, x, mean, rstd, w)
    x2, mean2, rstd2 = x.clone(), mean.clone(), rstd.clone()
    for i in (5, 7):
        x2[i], mean2[i], rstd2[i] = 0.0, 0.0, 1.0
    Z.zero_layernorm_bwd(dx2, None, None, dy, x2, mean2, rstd2, w)
    assert torch.equal(dx[good].view(torch.uint8), dx2[good].view(torch.uint8))
    assert bool(torch.isnan(dx[5]).all()) and bool(torch.isnan(dx[7]).all())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_weight_gradient_past_the_type(kind):
    """A weight gradient too large for binary16 is stored as inf."""
    rows, cols = 4096, 16
    dy = torch.full((rows, cols), 100.0, dtype=KINDS[kind], device="cuda")
    x = torch.randn(rows, cols, generator=gen("ovf")).to(KINDS[kind]).cuda()
    mean, rstd = _stats(x)
    db = torch.empty(cols, dtype=KINDS[kind], device="cuda")
    Z.zero_layernorm_bwd(torch.empty_like(x), None, db, dy, x, mean, rstd, None)
    assert bool((torch.isinf(db) if kind == "f16" else torch.isfinite(db)).all())     # 409600 > 65504


# ---- the joined form --------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_joined(rows, cols, kind):
    o = options(rows, cols, kind, "joined")
    log("joined", rows, cols, kind, o)
    g = gen("joined", rows, cols, kind)
    x = matrix(g, rows, cols, kind, 1.0, 0.2, pad=o["pad"], shift=o["shift"])
    res = matrix(g, rows, cols, kind, 2.0, pad=3, shift=1) if o["extra"] else None
    bias = vector(g, cols, o["vec"], 0.0, 0.3, 1) if o["extra"] else None
    w, b = vector(g, cols, o["vec"], 1.0, 0.3, o["shift"]), vector(g, cols, o["vec"], 0.0, 0.3)
    rng = rng_state(SEED, 3)
    r, y = empty(rows, cols, kind, pad=o["pad"], shift=o["shift"]), empty(rows, cols, kind, pad=1, shift=1)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    Z.zero_dropout_layernorm_fwd(r, y, mean, rstd, x, res, bias, w, b, EPS, o["p"], rng, 5)
    kept, s = O.keep(rows, cols, o["p"], SEED, 3, 5), O.scale(o["p"])
    same_bits(r, expect_r(x, res, bias, kept, s), "r")
    _check_fwd(r, y, mean, rstd, w, b, kind)
    assert canary_ok(r) and canary_ok(y)
    # backward, from the stored r and statistics
    dy = matrix(g, rows, cols, kind, 0.5, pad=o["pad"])
    dres = matrix(g, rows, cols, kind, 0.5, pad=8, shift=8) if o["extra"] else None
    dx, dr = empty(rows, cols, kind, pad=3, shift=o["shift"]), empty(rows, cols, kind, pad=o["pad"], shift=1)
    sums = [vector(g, cols, o["vec"], 0.5, 1.0, 1) for _ in range(3)]
    before = [f64(t) for t in sums]
    Z.zero_dropout_layernorm_bwd(dx, dr, *sums, dy, dres, r, mean, rstd, w, o["p"], rng, 5,
                                 accumulate=o["accumulate"], workspace=dirty_workspace(rows, cols))
    want, bound = O.norm_bwd(f64(dy), f64(r), f64(mean), f64(rstd), f64(w)[None], None if dres is None else f64(dres))
    e, e_e = want[0], 1.01 * bound[0]
    close(dr, e, O.stored(e_e, e, kind), "dr")
    d = O.dropped(e, kept, s)
    e_d = O.dropped(e_e, kept, s) + O.U * np.abs(d)
    close(dx, d, O.stored(e_d, d, kind), "dx")
    assert canary_ok(dx) and canary_ok(dr)
    assert bool((dx.cpu()[torch.from_numpy(~kept)] == 0).all())
    total, e_t = O.column_sum(d, e_d)
    for name, got, t, e, old in (("dw", sums[0], want[1], bound[1], before[0]), ("db", sums[1], want[2], bound[2], before[1]),
                                 ("dbias", sums[2], total, e_t, before[2])):
        if o["accumulate"]:
            t = t + old
            e = e + O.U * np.abs(t)
        close(got, t, O.stored(e, t, o["vec"]), name)


@pytest.mark.parametrize("rows,cols", [(1, 5), (37, 1600), (6, 8192), (3, 20011)])
def test_joined_equals_the_two_apart(rows, cols):
    """One pass gives the bits of the dropout followed by the layer norm."""
    log("joined = apart", rows, cols)
    g = gen("apart", rows, cols)
    x, res = matrix(g, rows, cols, "f16"), matrix(g, rows, cols, "f16", 2.0)
    bias, w, b = (vector(g, cols, "f16", a, 0.2) for a in (0.0, 1.0, 0.0))
    rng = rng_state(SEED, 0)
    r, y, r2, y2 = (torch.empty(rows, cols, dtype=torch.float16, device="cuda") for _ in range(4))
    st = [torch.empty(rows, device="cuda") for _ in range(4)]
    Z.zero_dropout_layernorm_fwd(r, y, st[0], st[1], x, res, bias, w, b, EPS, 0.2, rng, 9)
    Z.zero_dropout_fwd(r2, x, 0.2, rng, 9, residual=res, bias=bias)
    Z.zero_layernorm_fwd(y2, st[2], st[3], r2, w, b, EPS)
    same_bits(r, r2.cpu(), "r")
    same_bits(y, y2.cpu(), "y")
    same_bits(st[0], st[2].cpu(), "mean")
    same_bits(st[1], st[3].cpu(), "rstd")


@pytest.mark.parametrize("rows,cols", [(5, 40), (3, 600)])
def test_gradients_match_differences_of_the_forward_kernel(rows, cols):
    """The backward kernel against central differences of the forward kernel
    along random directions, in binary32.  With step h and unit direction the
    difference quotient is off by (h^2 / 6) f''' and by the forward's rounding
    over h.  Derived before the first run for these sizes: each y and r is off
    by at most ~ (d + 12) u times a value of order 3, so the loss, a sum of
    2 rows cols terms with random signs, by ~ 3 (d + 12) u sqrt(2 rows cols)
    (2e-3 at most here), over 2 h with h = 0.25 in the direction's own norm:
    under 4e-3; f''' of the normalised row along a unit direction is of order
    rstd^3 |c| / sqrt(cols), (h^2 / 6) f''' ~ 1e-2 |c|.  Both are compared with
    |gradient| ~ sqrt(rows cols): a tolerance of 2 percent of it covers them,
    and a wrong term of the formula shows as 10 percent and more."""
    log("differences", rows, cols)
    g = gen("diff", rows, cols)
    x, res = matrix(g, rows, cols, "f32"), matrix(g, rows, cols, "f32")
    bias, w, b = (vector(g, cols, "f32", a, 0.3) for a in (0.0, 1.0, 0.0))
    c, cr = torch.randn(rows, cols, generator=g).double().cuda(), torch.randn(rows, cols, generator=g).double().cuda()
    rng = rng_state(SEED, 0)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")

    def loss(x, res, bias, w, b):
        r, y = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
        Z.zero_dropout_layernorm_fwd(r, y, mean, rstd, x, res, bias, w, b, EPS, 0.25, rng, 1)
        return float((y.double() * c).sum() + (r.double() * cr).sum()), r

    base = [x.clone(), res.clone(), bias, w, b]
    _, r = loss(*base)
    dx, dr = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
    dw, db, dbias = (torch.empty(cols, device="cuda") for _ in range(3))
    Z.zero_dropout_layernorm_bwd(dx, dr, dw, db, dbias, c.float(), cr.float(), r, mean, rstd, w, 0.25, rng, 1)
    for i, grad in enumerate((dx, dr, dbias, dw, db)):
        norm = float(grad.double().norm())
        for k in range(3):                          # a random direction, and two with the gradient in them
            d = torch.randn(base[i].shape, generator=g).cuda()
            d = d / d.norm() + (0.0 if k == 0 else grad / norm)
            d = d / d.norm()
            v = [loss(*[t + s * 0.25 * d if j == i else t for j, t in enumerate(base)])[0] for s in (1, -1)]
            assert abs((v[0] - v[1]) / 0.5 - float((grad.double() * d.double()).sum())) <= 0.02 * norm + 4e-3, (i, k)


# ---- how they are called --------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("accumulate", [False, True])
def test_no_rows(kind, accumulate):
    """An empty batch: forward does nothing, the gradients are sums of nothing."""
    cols = 40
    x = torch.empty(0, cols, dtype=KINDS[kind], device="cuda")
    s = torch.empty(0, device="cuda")
    w = torch.ones(cols, device="cuda")
    rng = rng_state(SEED, 0)
    log("no rows", kind, accumulate)
    Z.zero_dropout_fwd(x, x, 0.1, rng)
    Z.zero_layernorm_fwd(x, s, s, x, w, w)
    Z.zero_dropout_layernorm_fwd(x, torch.empty_like(x), s, s, x, x, w, w, w, EPS, 0.1, rng)
    for call in (lambda t: Z.zero_dropout_bwd(x, x, 0.1, rng, dbias=t[2], accumulate=accumulate),
                 lambda t: Z.zero_layernorm_bwd(x, t[0], t[1], x, x, s, s, w, accumulate=accumulate),
                 lambda t: Z.zero_dropout_layernorm_bwd(x, torch.empty_like(x), *t, x, x, x, s, s, w, 0.1, rng,
                                                        accumulate=accumulate)):
        t = [torch.full((cols,), 5.0, device="cuda") for _ in range(3)]
        call(t)
        vals = {float(v) for u in t for v in u.cpu()}
        assert vals <= ({5.0} if accumulate else {0.0, 5.0})
    assert not any(float(v) for u in t for v in u.cpu()) or accumulate      # the joined call writes all three
    Z.zero_dropout_fwd(torch.empty(5, 0, dtype=KINDS[kind], device="cuda"),
                       torch.empty(5, 0, dtype=KINDS[kind], device="cuda"), 0.1, rng)


@pytest.mark.parametrize("rows,cols,kind", [(65, 1600, "bf16"), (3, 77, "bf16"), (4, 8192, "bf16"), (2, 20001, "bf16"),
                                            (5000, 1601, "f32"), (9000, 1100, "f16"), (700, 9001, "f32"), (4001, 5, "f16"),
                                            (20000, 333, "f32")])
def test_in_place(rows, cols, kind):
    """Outputs on the inputs' own memory give the same bits as apart."""
    log("in place", rows, cols, kind)
    g = gen("inplace", rows, cols)
    x, res = (matrix(g, rows, cols, kind).contiguous() for _ in range(2))
    dy, dres = (matrix(g, rows, cols, kind).contiguous() for _ in range(2))
    bias, w, b = (vector(g, cols, "f32", a, 0.3) for a in (0.0, 1.0, 0.0))
    rng = rng_state(SEED, 0)
    stats = lambda: [torch.empty(rows, device="cuda") for _ in range(2)]
    new = lambda: torch.empty_like(x)
    st, r, y = stats(), new(), new()
    Z.zero_dropout_layernorm_fwd(r, y, *st, x, res, bias, w, b, EPS, 0.3, rng, 2)
    dx, dr, sums = new(), new(), [torch.empty(cols, device="cuda") for _ in range(3)]
    Z.zero_dropout_layernorm_bwd(dx, dr, *sums, dy, dres, r, *st, w, 0.3, rng, 2)
    for r_on, y_on in (("x", "res"), ("res", "x"), ("res", None), (None, "x"), (None, "res")):
        a = {"x": x.clone(), "res": res.clone(), None: None}
        r2 = a[r_on] if r_on else new()
        y2 = a[y_on] if y_on else new()
        st2 = stats()
        Z.zero_dropout_layernorm_fwd(r2, y2, *st2, a["x"], a["res"], bias, w, b, EPS, 0.3, rng, 2)
        assert torch.equal(r2, r) and torch.equal(y2, y) and torch.equal(st2[0], st[0]) and torch.equal(st2[1], st[1])
    for dx_on, dr_on in (("dy", "dres"), ("dres", "dy"), ("r", "dy"), ("dy", "r"), (None, "dres")):
        a = {"dy": dy.clone(), "dres": dres.clone(), "r": r.clone()}
        dx2 = a[dx_on] if dx_on else new()
        s2 = [torch.empty(cols, device="cuda") for _ in range(3)]
        Z.zero_dropout_layernorm_bwd(dx2, a[dr_on], *s2, a["dy"], a["dres"], a["r"], *st, w, 0.3, rng, 2)
        assert torch.equal(dx2, dx) and torch.equal(a[dr_on], dr), (dx_on, dr_on)
        assert all(torch.equal(p, q) for p, q in zip(s2, sums))
    t = x.clone()
    Z.zero_layernorm_fwd(t, None, None, t, w, b, EPS)
    Z.zero_layernorm_fwd(y, None, None, x, w, b, EPS)
    assert torch.equal(t, y)
    t = x.clone()
    Z.zero_dropout_bwd(t, t, 0.3, rng, 2, dbias=sums[0])
    Z.zero_dropout_bwd(dx, x, 0.3, rng, 2, dbias=sums[1])
    assert torch.equal(t, dx) and torch.equal(sums[0], sums[1])


@pytest.mark.parametrize("rows,cols", [(5000, 1600), (900, 8192), (4097, 333)])
def test_equal_calls_give_equal_bits(rows, cols):
    log("repeat", rows, cols)
    g = gen("repeat", rows, cols)
    dy, r, dres = (matrix(g, rows, cols, "bf16") for _ in range(3))
    w = vector(g, cols, "f32", 1.0, 0.3)
    mean, rstd = _stats(r)
    rng = rng_state(SEED, 0)
    runs = []
    for _ in range(3):
        dx, dr = torch.empty_like(dy), torch.empty_like(dy)
        sums = [torch.empty(cols, device="cuda") for _ in range(3)]
        Z.zero_dropout_layernorm_bwd(dx, dr, *sums, dy, dres, r, mean, rstd, w, 0.1, rng, 0,
                                     workspace=dirty_workspace(rows, cols))
        runs.append([dx, dr, *sums])
    for other in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(runs[0], other))


def test_other_stream():
    """On a stream that is not the current one, the workspace from the
    allocator: the call waits for that stream's earlier work and the results
    are there once it is synchronised."""
    g = gen("stream")
    rows, cols = 2000, 1600
    dy0, r = matrix(g, rows, cols, "f16", 0.5), matrix(g, rows, cols, "f16")
    mean, rstd = _stats(r)
    w = vector(g, cols, "f16", 1.0, 0.3)
    want = [torch.empty_like(r), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")]
    Z.zero_layernorm_bwd(*want, dy0, r, mean, rstd, w)
    side = torch.cuda.Stream()
    got = [torch.empty_like(r), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")]
    dy = torch.zeros_like(dy0)
    torch.cuda.synchronize()
    log("other stream")
    with torch.cuda.stream(side):
        big = torch.empty(1 << 28, device="cuda")
        big.fill_(1.0)                              # work ahead of the input on that stream
        dy.copy_(dy0)
    Z.zero_layernorm_bwd(*got, dy, r, mean, rstd, w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once():
    """Two calls at once on two streams, each with its own workspace."""
    g = gen("two streams")
    rows, cols = 3000, 1600
    mats = [[matrix(g, rows, cols, "f16", 0.5), matrix(g, rows, cols, "f16")] for _ in range(2)]
    stats = [_stats(m[1]) for m in mats]
    out = lambda: [torch.empty(rows, cols, dtype=torch.float16, device="cuda"), torch.empty(cols, device="cuda"),
                   torch.empty(cols, device="cuda")]
    want = [out(), out()]
    for k in range(2):
        Z.zero_layernorm_bwd(*want[k], *mats[k], *stats[k], None)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [out(), out()]
    torch.cuda.synchronize()
    log("two streams")
    for _ in range(4):
        for k in range(2):
            Z.zero_layernorm_bwd(*got[k], *mats[k], *stats[k], None, stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[k], want[k]))


def test_graph_replays_draw_new_masks():
    """A training step's operators captured once: the generator's state lives in
    device memory and is advanced inside the graph, so every replay draws new
    masks; each is compared with the same calls made eagerly, with eager work
    and synchronisations between the replays.  Two graphs without a workspace
    of their own do not disturb each other."""
    g = gen("graph")
    rows, cols = 515, 1600
    x, res, dy = (matrix(g, rows, cols, "f16").contiguous() for _ in range(3))
    bias, w, b = (vector(g, cols, "f16", a, 0.2) for a in (0.0, 1.0, 0.0))

    class Body:
        def __init__(self, site):
            self.site, self.rng = site, rng_state(SEED, 0)
            self.r, self.y, self.dx, self.dr = (torch.zeros_like(x) for _ in range(4))
            self.st = [torch.zeros(rows, device="cuda") for _ in range(2)]
            self.sums = [torch.zeros(cols, dtype=torch.float16, device="cuda") for _ in range(3)]

        def step(self):
            Z.zero_dropout_layernorm_fwd(self.r, self.y, *self.st, x, res, bias, w, b, EPS, 0.1, self.rng, self.site)
            Z.zero_dropout_layernorm_bwd(self.dx, self.dr, *self.sums, dy, None, self.r, *self.st, w, 0.1, self.rng,
                                         self.site)
            Z.zero_rng_advance(self.rng)

        def outs(self):
            return [self.r, self.y, self.dx, self.dr, *self.st, *self.sums]

    eager, graphed = [Body(0), Body(1)], [Body(0), Body(1)]
    graphs = []
    for body in graphed:
        torch.cuda.synchronize()
        gr, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(gr, stream=side):
                body.step()
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(gr)
    torch.cuda.synchronize()
    assert Z.read_rng(graphed[0].rng).step == 0                 # capturing ran nothing
    last = None
    for k in range(5):
        log("graph replay", k)
        x.copy_(torch.randn(rows, cols, generator=g).half())
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        for body in eager:
            body.step()
        torch.cuda.synchronize()
        for e, c in zip(eager, graphed):
            assert all(torch.equal(p, q) for p, q in zip(e.outs(), c.outs()))
        mask = (graphed[0].dx == 0)
        assert last is None or not torch.equal(mask, last)
        last = mask
    assert Z.read_rng(graphed[0].rng).step == 5


# ---- sizes ------------------------------------------------------------------------------------------

def test_offsets_past_32_bits():
    """Rows 2^31 elements apart (in fp16, offsets past 2^32 bytes and, over the
    rows, past 2^32 elements)."""
    rows, cols, ld = 4, 1601, (1 << 31) + 7
    log("long offsets")
    buf = torch.zeros((rows - 1) * ld + cols, dtype=torch.float16, device="cuda")
    x = torch.as_strided(buf, (rows, cols), (ld, 1))
    g = gen("long")
    small = torch.randn(rows, cols, generator=g).half().cuda()
    x.copy_(small)
    w = vector(g, cols, "f32", 1.0, 0.3)
    rng = rng_state(SEED, 0)
    r, y = torch.empty_like(small), torch.empty_like(small)
    r2, y2 = torch.empty_like(small), torch.empty_like(small)
    st = [torch.empty(rows, device="cuda") for _ in range(2)]
    Z.zero_dropout_layernorm_fwd(r, y, *st, x, x, None, w, None, EPS, 0.2, rng)
    Z.zero_dropout_layernorm_fwd(r2, y2, None, None, small, small, None, w, None, EPS, 0.2, rng)
    assert torch.equal(r, r2) and torch.equal(y, y2)
    o = [[torch.empty(cols, device="cuda") for _ in range(3)] for _ in range(2)]
    dx, dr, dx2, dr2 = (torch.empty_like(small) for _ in range(4))
    x.copy_(r)
    Z.zero_dropout_layernorm_bwd(dx, dr, *o[0], x, x, x, *st, w, 0.2, rng)
    Z.zero_dropout_layernorm_bwd(dx2, dr2, *o[1], r, r, r, *st, w, 0.2, rng)
    assert torch.equal(dx, dx2) and torch.equal(dr, dr2) and all(torch.equal(a, b) for a, b in zip(*o))
    Z.zero_dropout_fwd(x, x, 0.2, rng, residual=x)              # stores through the long offsets too
    Z.zero_dropout_fwd(r2, r, 0.2, rng, residual=r)
    assert torch.equal(x, r2)


def test_more_groups_than_32_bits_count():
    """One column and more than 2^32 rows: every row is a group of its own, so
    the generator's counter passes 32 bits, and the grid goes around."""
    rows = (1 << 32) + 5
    x = torch.ones(rows, 1, dtype=torch.float16, device="cuda")
    log("2^32 groups")
    Z.zero_dropout_fwd(x, x, 0.5, rng_state(SEED, 1), 3)
    for first in (0, (1 << 30) - 50, (1 << 32) - 95):
        k = O.keep(100, 1, 0.5, SEED, 1, 3, first_row=first)
        assert np.array_equal(f64(x[first:first + 100]), k * 2.0), first


def test_very_wide_rows():
    """A flat tensor as one row of 2^30 columns, and sums over two rows of more
    columns than the fold's grid covers at once."""
    cols = 1 << 30
    log("one row of 2^30")
    x = torch.ones(1, cols, dtype=torch.float16, device="cuda")
    rng = rng_state(SEED, 1)
    Z.zero_dropout_fwd(x, x, 0.5, rng, 3)
    assert np.array_equal(f64(x[:, :800]), O.keep(1, 800, 0.5, SEED, 1, 3) * 2.0)
    out = O.philox4x32(((cols - 8) // 8, 0, 3, 1), (SEED & 0xFFFFFFFF, SEED >> 32))     # the last group
    want = [((int(o) >> s) & 0xFFFF) >= 32768 for o in out for s in (0, 16)]
    assert [bool(v) for v in x[0, -8:]] == want
    del x
    cols = (1 << 21) + 4099                          # past 65536 blocks of 32 columns
    log("two rows of 2^21 + 4099")
    dy = torch.randn(2, cols, device="cuda")
    db = torch.empty(cols, device="cuda")
    dx = torch.empty_like(dy)
    Z.zero_dropout_bwd(dx, dy, 0.25, rng, 3, dbias=db)
    assert torch.equal(db, dx[0] + dx[1])
    w = torch.rand(cols, device="cuda") + 0.5
    y, st = torch.empty_like(dy), [torch.empty(2, device="cuda") for _ in range(2)]
    Z.zero_layernorm_fwd(y, *st, dy, w, None, EPS)
    _check_fwd(dy, y, *st, w, None, "f32")


@pytest.mark.parametrize("rows,cols", [((1 << 20) + 77, 8), (70_001, 24)])
def test_many_rows(rows, cols):
    """More rows than a launch has workgroups."""
    log("many rows", rows, cols)
    x = torch.randn(rows, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    dy = torch.randn(rows, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    y, st = torch.empty_like(x), [torch.empty(rows, device="cuda") for _ in range(2)]
    Z.zero_layernorm_fwd(y, *st, x, None, None, EPS)
    _check_fwd(x, y, *st, None, None, "f32")
    dx, dw, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    Z.zero_layernorm_bwd(dx, dw, db, dy, x, *st, None)
    want, bound = O.norm_bwd(f64(dy), f64(x), f64(st[0]), f64(st[1]), np.ones((1, cols)), None)
    close(dx, want[0], O.stored(bound[0], want[0], "f32"), "dx")
    close(dw, want[1], O.stored(bound[1], want[1], "f32"), "dw")
    close(db, want[2], O.stored(bound[2], want[2], "f32"), "db")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cols", [9, 100, 255, 300, 511, 700, 1024, 1100, 2048, 2500, 3500, 5120, 6000, 7000, 8191, 8193, 10000,
                                  12000, 15000, 16384, 16385])
def test_every_width_class(cols, kind):
    """Each number of threads a row can have, in the forward and backward
    passes, with more rows than one workgroup holds."""
    rows = 5 if cols > 1000 else 150
    log("width", cols, kind)
    g = gen("width", cols, kind)
    x, res = matrix(g, rows, cols, kind, 1.0, 0.2), matrix(g, rows, cols, kind, 2.0, pad=1)
    bias, w, b = vector(g, cols, "f32", 0.0, 0.3), vector(g, cols, "f32", 1.0, 0.3), vector(g, cols, "f32", 0.0, 0.3)
    rng = rng_state(SEED, 1)
    r, y = empty(rows, cols, kind), empty(rows, cols, kind, pad=2)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    Z.zero_dropout_layernorm_fwd(r, y, mean, rstd, x, res, bias, w, b, EPS, 0.25, rng, 2)
    kept, s = O.keep(rows, cols, 0.25, SEED, 1, 2), O.scale(0.25)
    same_bits(r, expect_r(x, res, bias, kept, s), "r")
    _check_fwd(r, y, mean, rstd, w, b, kind)
    y2, m2, s2 = empty(rows, cols, kind), torch.empty_like(mean), torch.empty_like(rstd)
    Z.zero_layernorm_fwd(y2, m2, s2, r, w, b, EPS)
    _check_fwd(r, y2, m2, s2, w, b, kind)
    dy, dres = matrix(g, rows, cols, kind, 0.5), matrix(g, rows, cols, kind, 0.5)
    dx, dr = empty(rows, cols, kind, pad=1), empty(rows, cols, kind)
    sums = [torch.empty(cols, device="cuda") for _ in range(3)]
    Z.zero_dropout_layernorm_bwd(dx, dr, *sums, dy, dres, r, mean, rstd, w, 0.25, rng, 2,
                                 workspace=dirty_workspace(rows, cols))
    want, bound = O.norm_bwd(f64(dy), f64(r), f64(mean), f64(rstd), f64(w)[None], f64(dres))
    e, e_e = want[0], 1.01 * bound[0]
    close(dr, e, O.stored(e_e, e, kind), "dr")
    d = O.dropped(e, kept, s)
    e_d = O.dropped(e_e, kept, s) + O.U * np.abs(d)
    close(dx, d, O.stored(e_d, d, kind), "dx")
    close(sums[0], want[1], O.stored(bound[1], want[1], "f32"), "dw")
    close(sums[1], want[2], O.stored(bound[2], want[2], "f32"), "db")
    t, e_t = O.column_sum(d, e_d)
    close(sums[2], t, O.stored(e_t, t, "f32"), "dbias")
    dx2, dw2 = empty(rows, cols, kind), torch.empty(cols, device="cuda")
    Z.zero_layernorm_bwd(dx2, dw2, None, dy, r, mean, rstd, w, dres=dres, workspace=dirty_workspace(rows, cols))
    close(dx2, e, O.stored(e_e, e, kind), "dx of the layer norm alone")
    close(dw2, want[1], O.stored(bound[1], want[1], "f32"), "dw of the layer norm alone")


@pytest.mark.parametrize("rows,cols,kind", [(36000, 1601, "f16"), (36000, 1600, "bf16"), (300_001, 70, "f32"),
                                            (7000, 8192, "f16"), (9_000_001, 3, "f32"), (2100, 12001, "f32")])
def test_past_the_cache(rows, cols, kind):
    """Calls that move more than the cache holds (their loads take the other
    hint, and a workgroup many blocks of rows): the first, middle and last
    rows against the 64-bit forms, the sums over all rows against sums in 64
    bits on the device."""
    log("past the cache", rows, cols, kind)
    gg = torch.Generator("cuda")
    gg.manual_seed(rows + cols)
    make = lambda s: (torch.randn(rows, cols, device="cuda", generator=gg) * s).to(KINDS[kind])
    x, res, dy, dres = make(1.0), make(2.0), make(0.5), make(0.5)
    g = gen("past", rows, cols)
    bias, w, b = vector(g, cols, "f32", 0.0, 0.3), vector(g, cols, "f32", 1.0, 0.3), vector(g, cols, "f32", 0.0, 0.3)
    rng = rng_state(SEED, 1)
    r, y, out, dx, dr = (torch.empty_like(x) for _ in range(5))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    Z.zero_dropout_layernorm_fwd(r, y, mean, rstd, x, res, bias, w, b, EPS, 0.25, rng, 2)
    Z.zero_dropout_fwd(out, x, 0.25, rng, 2, residual=res, bias=bias)
    assert torch.equal(out, r)
    y2 = torch.empty_like(x)
    Z.zero_layernorm_fwd(y2, None, None, r, w, b, EPS)
    assert torch.equal(y2, y)
    sums = [torch.empty(cols, device="cuda") for _ in range(3)]
    Z.zero_dropout_layernorm_bwd(dx, dr, *sums, dy, dres, r, mean, rstd, w, 0.25, rng, 2,
                                 workspace=dirty_workspace(rows, cols))
    s = O.scale(0.25)
    for first in (0, rows // 2, rows - 40):
        at = slice(first, first + 40)
        kept = O.keep(40, cols, 0.25, SEED, 1, 2, first_row=first)
        same_bits(r[at], expect_r(x[at], res[at], bias, kept, s), "r")
        _check_fwd(r[at], y[at], mean[at], rstd[at], w, b, kind)
        want, bound = O.norm_bwd(f64(dy[at]), f64(r[at]), f64(mean[at]), f64(rstd[at]), f64(w)[None], f64(dres[at]))
        e, e_e = want[0], 1.01 * bound[0]
        close(dr[at], e, O.stored(e_e, e, kind), "dr")
        d = O.dropped(e, kept, s)
        close(dx[at], d, O.stored(O.dropped(e_e, kept, s) + O.U * np.abs(d), d, kind), "dx")
    # sums: d = rows / 256 + 40 additions in a chain is still far above what a column takes; bounded by all of them
    chain = (rows + 32.0) * O.U
    h = (r.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for name, got, term in (("dw", sums[0], dy.double() * h), ("db", sums[1], dy.double())):
        close(got, f64(term.sum(0)), f64(term.abs().sum(0)) * min(chain, 1e-3) + 1e-30, name)
    del h
    # dbias: the stored dx is off by half a step of its type from what is summed
    t = dx.double()
    close(sums[2], f64(t.sum(0)), f64(t.abs().sum(0)) * (min(chain, 1e-3) + 1.01 * O.half_step(kind)) + 1e-30, "dbias")
    # the other backward passes over the same rows
    Z.zero_layernorm_bwd(y2, sums[0], sums[1], dy, r, mean, rstd, w, dres=dres)
    same = (y2 == dr) | ((y2.float() - dr.float()).abs() <= dr.float().abs() * 4 * O.half_step(kind) + 1e-6)
    assert bool(same.all())
    t = out
    Z.zero_dropout_bwd(t, dy, 0.25, rng, 2, dbias=sums[2])
    close(sums[2], f64(t.double().sum(0)), f64(t.double().abs().sum(0)) * (min(chain, 1e-3) + 1.01 * O.half_step(kind))
          + 1e-30, "dbias of dropout alone")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_subnormal_values(kind):
    """Values below the type's smallest normal one go through as they are (no
    flush to zero on any path)."""
    rows, cols = 7, 333
    g = gen("subnormal", kind)
    tiny = {"f16": 2.0 ** -20, "bf16": 2.0 ** -130}[kind]
    x, dy = matrix(g, rows, cols, kind, tiny), matrix(g, rows, cols, kind, tiny)
    out = empty(rows, cols, kind)
    log("subnormal", kind)
    Z.zero_dropout_fwd(out, x, 0.5, rng_state(SEED, 0), 1, residual=dy)
    same_bits(out, expect_r(x, dy, None, O.keep(rows, cols, 0.5, SEED, 0, 1), 2.0), "out")
    r = matrix(g, rows, cols, kind, 1.0)
    mean, rstd = _stats(r)
    dx, db = empty(rows, cols, kind), torch.empty(cols, device="cuda")
    Z.zero_layernorm_bwd(dx, None, db, dy, r, mean, rstd, None)
    want, bound = O.norm_bwd(f64(dy), f64(r), f64(mean), f64(rstd), np.ones((1, cols)), None)
    close(dx, want[0], O.stored(bound[0] + 2.0 ** -149 * cols, want[0], kind), "dx")
    close(db, want[2], O.stored(bound[2], want[2], "f32"), "db")
