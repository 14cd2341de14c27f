"""The sums over the rows (dw, db, dbias) held exactly.  Inputs are whole
numbers chosen so that every value that enters a sum is a whole number and
every partial sum stays below 2^24: then binary32 sums are exact in any order,
and what the kernels give has to be equal, not close.  Shapes give a workgroup
several blocks of rows (more than the rows it keeps in flight) and leave the
last one short.

The rows come in pairs of columns, (2k, 2k + 1), with equal x and opposite dy,
so sum(g) = sum(g h) = 0 and the gradient at x is g + dres, a whole number too.
A mean of 0 and an rstd of 1 are handed in; the dropout's factor is 2."""
import zlib

import numpy as np
import pytest
import torch

import layer_oracle as O

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402

KINDS = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SEED = 0x5EED5EED12345


def log(*a):
    print("[sums]", *a, flush=True)


def whole(g, rows, cols, most, kind):
    """Whole numbers in [-most, most] on the device."""
    return torch.randint(-most, most + 1, (rows, cols), generator=g, device="cuda", dtype=torch.int8).to(KINDS[kind])


def inputs(rows, cols, kind):
    g = torch.Generator("cuda")
    g.manual_seed(zlib.crc32(repr((rows, cols, kind)).encode()))
    x, dy, dres = (whole(g, rows, cols, 3, kind) for _ in range(3))
    even = cols // 2 * 2
    x[:, 1:even:2] = x[:, 0:even:2]
    dy[:, 1:even:2] = -dy[:, 0:even:2]
    if cols % 2:
        dy[:, -1] = 0                               # the column without a partner
    return x, dy, dres


def kept_rows(rows, cols, step, site):
    """The kept elements as 0 and 1 on the device, a slice of rows at a time."""
    out = torch.empty(rows, cols, dtype=torch.bool, device="cuda")
    at_once = max(1, (1 << 23) // cols)
    for first in range(0, rows, at_once):
        k = O.keep(min(at_once, rows - first), cols, 0.5, SEED, step, site, first_row=first)
        out[first:first + k.shape[0]] = torch.from_numpy(k).cuda()
    return out


def column_sums(terms, pieces):
    """The sums over the rows in 64 bits, and the smallest magnitude that a
    wrong result would be off by at its worst column, if one of `pieces`
    blocks of rows were missing, or all of them."""
    total = torch.zeros(terms.shape[1], dtype=torch.float64, device="cuda")
    least = float("inf")
    for part in terms.split(-(-terms.shape[0] // pieces)):
        s = part.double().sum(0)
        total += s
        least = min(least, float(s.abs().max()))
    assert float(total.abs().max()) < 2 ** 24
    return total, min(least, float(total.abs().max()))


def check(name, got, terms, pieces=16):
    want, least = column_sums(terms, pieces)
    assert least > 0, f"{name}: the inputs would not show a missing block of rows"
    assert torch.equal(got.double(), want), (name, int((got.double() != want).sum()), float((got.double() - want).abs().max()))


# rows x cols: at least three blocks of rows a workgroup and a short last one, for every number of threads a row;
# 1585 x 1600 on the smaller grid that short batches take; past 8192 columns several rows to each strip's workgroup
ONE_PASS = [(787_003, 5), (164_429, 24), (99_331, 100), (50_021, 250), (25_013, 333), (13_001, 1000), (7_575, 1600),
            (1_585, 1600), (3_101, 4000), (1_155, 8192)]
WIDE = [(617, 8200), (613, 9001), (458, 20_001)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", ONE_PASS + WIDE)
def test_sums_are_exact(rows, cols, kind):
    log(rows, cols, kind)
    x, dy, dres = inputs(rows, cols, kind)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    new = lambda: torch.full((cols,), float("nan"), device="cuda")
    ws = lambda: torch.full((Z.zero_layer_workspace_bytes(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    # layer norm
    dx, dw, db = torch.empty_like(x), new(), new()
    Z.zero_layernorm_bwd(dx, dw, db, dy, x, mean, rstd, None, dres=dres, workspace=ws())
    assert torch.equal(dx, dy + dres)
    check("dw", dw, dy * x)
    check("db", db, dy)
    # dropout with its bias gradient
    rng = torch.zeros(Z.RNG_BYTES, dtype=torch.uint8, device="cuda")
    Z.zero_rng_init(rng, SEED)
    kept = kept_rows(rows, cols, 0, 6)
    dbias = new()
    Z.zero_dropout_bwd(dx, dres, 0.5, rng, 6, dbias=dbias, workspace=ws())
    want = torch.where(kept, 2 * dres, 0)
    assert torch.equal(dx, want)
    check("dbias", dbias, want)
    # the joined form
    dr, dw, db, dbias = torch.empty_like(x), new(), new(), new()
    Z.zero_dropout_layernorm_bwd(dx, dr, dw, db, dbias, dy, dres, x, mean, rstd, None, 0.5, rng, 6, workspace=ws())
    e = dy + dres
    want = torch.where(kept, 2 * e, 0)
    assert torch.equal(dr, e) and torch.equal(dx, want)
    check("joined dw", dw, dy * x)
    check("joined db", db, dy)
    check("joined dbias", dbias, want)
    # added to what is there
    before = [t.clone() for t in (dw, db, dbias)]
    Z.zero_dropout_layernorm_bwd(dx, dr, dw, db, dbias, dy, dres, x, mean, rstd, None, 0.5, rng, 6, accumulate=True,
                                 workspace=ws())
    assert all(torch.equal(a, 2 * b) for a, b in zip((dw, db, dbias), before))


@pytest.mark.parametrize("rows,cols,kind", [(36_001, 1601, "f16"), (36_001, 1601, "f32"), (6_500, 8192, "bf16"),
                                            (2_100, 12_001, "f32"), (1_300_003, 24, "bf16")])
def test_sums_are_exact_past_the_cache(rows, cols, kind):
    """The same where a call moves more than the cache holds (the other loads)."""
    test_sums_are_exact(rows, cols, kind)


def test_a_missing_block_would_show():
    """What `check` compares with, with a block of rows taken out of the
    gradient that it is given, or with zeros: it does not pass."""
    x, dy, _ = inputs(7_575, 1600, "f16")
    good = dy.double().sum(0)
    check("db", good, dy)
    for bad in (torch.zeros_like(good), good - dy[:4].double().sum(0), good - dy[-3:].double().sum(0)):
        with pytest.raises(AssertionError):
            check("db", bad, dy)


# ---- no rows -----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("cols", [3, 40, 9001])
def test_sums_of_no_rows(kind, accumulate, cols):
    """An empty batch: each call stores 0 to (or, accumulating, leaves) the
    gradients it has, and touches no other."""
    log("no rows", kind, accumulate, cols)
    x, s = torch.empty(0, cols, dtype=KINDS[kind], device="cuda"), torch.empty(0, device="cuda")
    rng = torch.zeros(Z.RNG_BYTES, dtype=torch.uint8, device="cuda")
    Z.zero_rng_init(rng, SEED)
    calls = {
        (2,): lambda t: Z.zero_dropout_bwd(x, x, 0.1, rng, dbias=t[2], accumulate=accumulate),
        (0, 1): lambda t: Z.zero_layernorm_bwd(x, t[0], t[1], x, x, s, s, None, accumulate=accumulate),
        (0,): lambda t: Z.zero_layernorm_bwd(x, t[0], None, x, x, s, s, None, accumulate=accumulate),
        (0, 1, 2): lambda t: Z.zero_dropout_layernorm_bwd(x, torch.empty_like(x), *t, x, x, x, s, s, None, 0.1, rng,
                                                          accumulate=accumulate),
        (1, 2): lambda t: Z.zero_dropout_layernorm_bwd(x, torch.empty_like(x), None, t[1], t[2], x, x, x, s, s, None, 0.1,
                                                       rng, accumulate=accumulate)}
    for own, call in calls.items():
        t = [torch.full((cols,), 5.0, device="cuda") for _ in range(3)]
        call(t)
        for i in range(3):
            want = 5.0 if accumulate or i not in own else 0.0
            assert bool((t[i] == want).all()), (own, i)
