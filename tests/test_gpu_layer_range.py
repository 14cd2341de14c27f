"""The norms' backward passes over the range of binary32 and bfloat16: rows of
a spread whose reciprocal squared, or whose reciprocal times the gradient, is
below or above what binary32 holds, where the gradients themselves are well
inside it, against the 64-bit forms, within their bounds.  And dropout over
more groups than one launch has threads."""
import zlib

import numpy as np
import pytest
import torch

import layer_oracle as O

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402

KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}
SEED = 0x0F1E2D3C4B5A6978

# What binary32 loses where a result or a product near it is subnormal: half
# of its smallest step for each of the last two roundings of e.
FLOOR = 2.0 ** -149


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, want, bound, what):
    bad = ~(np.abs(f64(got) - want) <= bound)
    if bad.any():
        i = tuple(int(k[0]) for k in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first at {i}: got {f64(got)[i]!r}, "
                             f"want {want[i]!r}, bound {np.broadcast_to(bound, want.shape)[i]!r}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cols", [5, 64, 1600, 8192, 9001])
@pytest.mark.parametrize("spread,scale", [(1e17, 1e-9), (1e18, 1e-6), (1e18, 1e-12), (1e17, 1e-30), (1e-21, 1.0)])
def test_backward_over_the_range(kind, cols, spread, scale):
    rows = 6
    print("[range]", kind, cols, spread, scale, flush=True)
    g = torch.Generator()
    g.manual_seed(zlib.crc32(repr((kind, cols, spread, scale)).encode()))
    draw = lambda *shape: torch.randn(*shape, generator=g, dtype=torch.float64)
    r = ((draw(rows, cols) + 0.3) * spread).to(KINDS[kind])
    mean = r.double().mean(1).float()
    rstd = r.double().var(1, unbiased=False).rsqrt().float()
    h = (r.double() - mean.double()[:, None]) * rstd.double()[:, None]
    dy = ((0.7 * h + 0.5 * draw(rows, cols)) * scale).to(KINDS[kind])     # along h: sum(g h) does not vanish
    dres = (draw(rows, cols) * (scale / spread)).to(KINDS[kind])
    w = 1.0 + 0.3 * draw(cols).float()
    r, mean, rstd, dy, dres, w = (t.cuda() for t in (r, mean, rstd, dy, dres, w))
    want, bound = O.norm_bwd(f64(dy), f64(r), f64(mean), f64(rstd), f64(w)[None], None)
    dx, dw, db = torch.empty_like(r), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    Z.zero_layernorm_bwd(dx, dw, db, dy, r, mean, rstd, w)
    close(dx, want[0], O.stored(bound[0] + FLOOR, want[0], kind), "dx")
    close(dw, want[1], O.stored(bound[1], want[1], "f32"), "dw")
    close(db, want[2], O.stored(bound[2], want[2], "f32"), "db")
    # the joined form, with the residual stream's gradient; p = 1/2: the factor 2 is exact
    want, bound = O.norm_bwd(f64(dy), f64(r), f64(mean), f64(rstd), f64(w)[None], f64(dres))
    rng = torch.zeros(Z.RNG_BYTES, dtype=torch.uint8, device="cuda")
    Z.zero_rng_init(rng, SEED)
    dx, dr, dbias = torch.empty_like(r), torch.empty_like(r), torch.empty(cols, device="cuda")
    Z.zero_dropout_layernorm_bwd(dx, dr, dw, db, dbias, dy, dres, r, mean, rstd, w, 0.5, rng, 3)
    kept = O.keep(rows, cols, 0.5, SEED, 0, 3)
    e, e_e = want[0], 1.01 * bound[0] + FLOOR
    close(dr, e, O.stored(e_e, e, kind), "dr")
    d, e_d = O.dropped(e, kept, 2.0), O.dropped(e_e, kept, 2.0)
    close(dx, d, O.stored(e_d, d, kind), "joined dx")
    close(dw, want[1], O.stored(bound[1], want[1], "f32"), "joined dw")
    close(db, want[2], O.stored(bound[2], want[2], "f32"), "joined db")
    total, e_t = O.column_sum(d, e_d)
    close(dbias, total, O.stored(e_t, total, "f32"), "dbias")


@pytest.mark.parametrize("rows,cols,kind", [((1 << 29) + 41, 9, "f16"), ((1 << 29) + 41, 9, "f32"),
                                            ((1 << 22) + 3, 2050, "bf16"), ((1 << 22) + 3, 2050, "f32")])
def test_dropout_past_one_launch(rows, cols, kind):
    """More groups of 8 columns than the threads of a launch: the grid goes
    around.  In place, with a residual and a bias, rows of few groups and of
    more than a workgroup's threads, an odd width and an even one; p = 1/2 and
    whole numbers, so every value is exact."""
    groups = -(-cols // 8)
    assert rows * groups > 1 << 30
    print("[range] past one launch", rows, cols, kind, flush=True)
    x = torch.ones(rows, cols, dtype={"f16": torch.float16, **KINDS}[kind], device="cuda")
    bias = (torch.arange(cols) % 5).float().cuda()
    rng = torch.zeros(Z.RNG_BYTES, dtype=torch.uint8, device="cuda")
    Z.zero_rng_init(rng, SEED)
    Z.zero_dropout_fwd(x, x, 0.5, rng, 8, residual=x, bias=bias)
    most = 3.0 + 2.0 * bias                                       # 1 + 2 (1 + bias) where kept, else 1
    around = (1 << 30) // groups                                  # where the second round begins
    for first in (0, 1234567, around - 50, around, rows - 100):
        kept = torch.from_numpy(O.keep(100 if first + 100 <= rows else rows - first, cols, 0.5, SEED, 0, 8, first_row=first))
        want = torch.where(kept, most.cpu(), 1.0)
        assert torch.equal(x[first:first + kept.shape[0]].float().cpu(), want), first
    for part in x.split(1 << 26 if cols < 100 else 1 << 18):      # every element was written, once
        v = part.float()
        assert bool(((v == 1.0) | (v == most)).all())
