"""Norms of queries and keys with the rotation on the GPU against the 64-bit
forms, within bounds derived from the roundings."""
import math

import pytest
import torch

import attention_oracle as A
from test_gpu_attention import BF16, F16, F32, SENTINEL, close, normal, strided, untouched

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402

EPS, BASE = 1e-6, 10000.0


def log(*a):
    print("[qk]", *a, flush=True)


def run(tokens, heads, kv_heads, dim, dtype, rot=None, interleaved=False, wtype=None, weights=True, layout="plain", positions=None, period=0,
        in_place=False, accumulate=False, gtype=None, spread=1.0):
    rot = dim if rot is None else rot
    log(tokens, heads, kv_heads, dim, dtype, rot, interleaved, layout)
    g = torch.Generator().manual_seed(tokens * 1000 + dim)
    wtype = wtype or dtype
    pos = torch.arange(tokens) % period if period else torch.arange(tokens)
    if positions is not None:
        pos = positions
    rows = int(pos.max()) + 1 if tokens else 1
    table = torch.full((rows, rot // 2, 2), SENTINEL, device="cuda") if rot else None
    if rot:
        Z.zero_rope_table(table, BASE)
    cs = A.angles(pos, rot, BASE) if rot else None
    dev_pos = None if positions is None else positions.int().cuda()
    x = [normal(g, tokens, h, dim, dtype=dtype, scale=spread) for h in (heads, kv_heads)]
    dy = [normal(g, tokens, h, dim, dtype=dtype, scale=0.1) for h in (heads, kv_heads)]
    w = [(1.0 + 0.3 * torch.randn(dim, generator=g, dtype=torch.float64)).to(wtype) if weights else None for _ in range(2)]
    w64 = [torch.ones(dim, dtype=torch.float64) if v is None else v.double() for v in w]
    dw_ = [None if v is None else v.cuda() for v in w]
    sides = 2 if kv_heads else 1

    def place(ts):
        out = []
        for t in ts[:sides]:
            buf, view = strided(*t.shape, t.dtype, layout)
            view.copy_(t)
            out.append((buf, view))
        return out + [(None, None)] * (2 - sides)

    xs = place(x)
    outs = xs if in_place else place([torch.full_like(t, SENTINEL) for t in x])
    kw = dict(positions=dev_pos, period=period, interleaved=interleaved)
    Z.zero_qk_norm_rope_fwd(outs[0][1], outs[1][1], xs[0][1], xs[1][1], dw_[0], dw_[1] if kv_heads else None, table, EPS, **kw)
    torch.cuda.synchronize()
    for i in range(sides):
        want, e = A.qk_fwd(x[i].double(), w64[i], cs, EPS, interleaved)
        # the table's angles are rounded once: half a step of 1
        e = e + (2 * A.U * (x[i].double() * (x[i].double().square().mean(2, keepdim=True) + EPS).rsqrt() * w64[i]).abs().amax(2, keepdim=True) if rot else 0)
        close(outs[i][1], want, A.stored(e, want, dtype), f"y{i}")
        assert untouched(*outs[i])

    xs, gs = place(x), place(dy)
    outs = gs if in_place else place([torch.full_like(t, SENTINEL) for t in x])
    gtype = gtype or wtype
    start = 2.5 if accumulate else 0.0
    grads = [torch.full((dim,), start if accumulate else SENTINEL, dtype=gtype, device="cuda") if weights else None for _ in range(sides)]
    grads += [None] * (2 - sides)
    Z.zero_qk_norm_rope_bwd(outs[0][1], outs[1][1], grads[0], grads[1], gs[0][1], gs[1][1], xs[0][1], xs[1][1], dw_[0],
                            dw_[1] if kv_heads else None, table, EPS, accumulate=accumulate, **kw)
    torch.cuda.synchronize()
    for i in range(sides):
        (dx, dw), (e_dx, e_dw) = A.qk_bwd(dy[i].double(), x[i].double(), w64[i], cs, EPS, interleaved)
        if rot:                                      # of the table's rounding, through every product of dy
            rstd = (x[i].double().square().mean(2, keepdim=True) + EPS).rsqrt()
            h = (x[i].double() * rstd).abs()
            one = 2 * A.U * dy[i].double().abs().amax(2, keepdim=True) * torch.ones(dim)
            gw = one * w64[i].abs()
            e_dx = e_dx + rstd * (gw + h * (gw * h).mean(2, keepdim=True))
            e_dw = e_dw + (one * h).sum((0, 1))
        close(outs[i][1], dx, A.stored(e_dx, dx, dtype), f"dx{i}")
        assert untouched(*outs[i])
        if weights:
            close(grads[i], dw + start, A.stored(e_dw + 2 * A.U * (dw.abs() + start), dw + start, gtype), f"dw{i}")


@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("dim", [2, 8, 10, 16, 20, 32, 48, 64, 80, 96, 120, 128, 192, 250, 256])
def test_dims(dim, dtype):
    for interleaved in (False, True):
        for rot in {dim, 0, dim // 4 * 2, min(dim, 16)}:
            run(37, 5, 2, dim, dtype, rot, interleaved)


@pytest.mark.parametrize("tokens,heads,kv_heads", [(1, 1, 1), (1, 25, 25), (3, 64, 8), (1000, 25, 25), (257, 7, 0), (2, 1, 0)])
def test_shapes(tokens, heads, kv_heads):
    for dtype in (F16, F32):
        run(tokens, heads, kv_heads, 64, dtype)
        run(tokens, heads, kv_heads, 36, dtype, 20)


@pytest.mark.parametrize("layout", ["joint", "odd", "heads"])
def test_layouts(layout):
    for dim in (64, 44):
        for in_place in (False, True):
            run(50, 3, 2, dim, F16, layout=layout, in_place=in_place)
            run(50, 3, 2, dim, F32, layout=layout, in_place=in_place, interleaved=True)


def test_weights():
    for gtype in (BF16, F32):
        run(60, 4, 2, 64, BF16, wtype=F32, gtype=gtype)
        run(60, 4, 2, 64, BF16, gtype=gtype, accumulate=True)
        run(60, 4, 2, 30, BF16, 10, wtype=F32, gtype=gtype, accumulate=True)
    run(60, 4, 2, 64, F16, weights=False)
    run(60, 4, 2, 22, F16, weights=False)


def test_positions():
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 5000, (97,), generator=g)
    for dim in (64, 34):
        run(97, 3, 1, dim, F32, positions=pos)
        run(97, 3, 1, dim, F16, period=10)


def test_sizes_of_rows():
    """Heads whose squares leave binary16 or vanish beside eps."""
    for spread in (1e-4, 200.0):
        run(40, 3, 2, 64, F16, spread=spread)
        run(40, 3, 2, 64, BF16, spread=spread * spread)


def test_far_angles():
    """Positions up to 2^20: the table is formed in binary64."""
    n = 1 << 20
    table = torch.empty(n + 1, 8, 2, device="cuda")
    Z.zero_rope_table(table, BASE)
    at = torch.tensor([0, 1, 2, 1000, 65535, 99999, n - 1, n])
    want = A.angles(at, 16, BASE)
    close(table[at.cuda()], want, 2.0 ** -24 + 1e-9 + 0 * want, "table")


def test_positions_outside_the_table_give_nan():
    table = torch.empty(10, 32, 2, device="cuda")
    Z.zero_rope_table(table)
    for dim in (64, 66):
        x = torch.randn(5, 2, dim, device="cuda")
        pos = torch.tensor([0, 9, 10, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        y = torch.empty_like(x)
        Z.zero_qk_norm_rope_fwd(y, None, x, None, None, None, table, positions=pos)
        bad = y.isnan().flatten(1)
        assert not bool(bad[:2].any()) and bool(bad[2:, :64].any(1).all())
        assert bool(y[2:, :, :64].isnan().all()) and not bool(y[2:, :, 64:].isnan().any())
