"""binary16's exponents in the attention kernels: values as large as binary16
holds, whose gradients fit, and keys with weights far below the row's largest,
which are many."""
import math

import pytest
import torch

import attention_oracle as A
from test_gpu_attention import BF16, F16, Call, close

pytestmark = pytest.mark.gpu


def log(*a):
    print("[units]", *a, flush=True)


class LargeValues(Call):
    """Rows `at` of v up to binary16's largest values, along dout and against it in turn; dout small enough for gradients that
    fit."""

    def __init__(self, *args, at=slice(None), size=30000.0, **kw):
        super().__init__(*args, do_scale=1e-3, **kw)
        sign = 1.0 - 2.0 * (torch.arange(self.tokens) % 2)[:, None, None]
        self.v[at] = ((0.5 + self.v.double().abs()) * sign * size).clamp(-65504.0, 65504.0).to(self.dtype)[at]
        self.do.abs_()
        self.d["v"].copy_(self.v)
        self.d["do"].copy_(self.do)


@pytest.mark.parametrize("size", [100.0, 1000.0, 30000.0, 1e6])
def test_large_values(size):
    """ds may leave binary16 in units of |do|, by up to 2 |v|; what it gives at the queries and keys does not."""
    for dim in (64, 128):
        log("large values", size, dim)
        c = LargeValues([300, 40], 2, 1, dim, F16, size=size)
        got = c.check_bwd(*c.check_fwd())
        assert all(bool(t.isfinite().all()) for t in got[:3])


@pytest.mark.parametrize("dim", [8, 24, 40, 72, 80, 120])
def test_large_values_at_other_head_sizes(dim):
    for layout in ("plain", "joint", "odd", "heads"):
        log("large values", dim, layout)
        c = LargeValues([90, 1, 150], 4, 2, dim, F16, window=40, sinks=3, layout=layout, size=60000.0, after=2)
        got = c.check_bwd(*c.check_fwd())
        assert all(bool(t[:c.end].isfinite().all()) for t in got[:3])


@pytest.mark.parametrize("starts", [[0, 1, 20], [0, 3, 601]])
def test_large_values_with_a_bias(starts):
    """The gradient of the bias takes each ds once."""
    for dim in (64, 128):
        log("large values, bias", starts, dim)
        c = LargeValues([300, 40], 2, 2, dim, F16, starts=starts, bias_dtype=torch.float32)
        got = c.check_bwd(*c.check_fwd())
        assert all(bool(t.isfinite().all()) for t in got)


def test_large_values_of_the_first_tokens():
    """Queries long behind the window, taken apart; many query heads a key head; rows off 16-byte places."""
    for lengths, heads, kv, dim, layout in (([2500], 2, 1, 64, "plain"), ([1400, 30], 8, 1, 128, "plain"), ([1300], 2, 2, 64, "odd")):
        log("large values, first tokens", lengths, dim)
        c = LargeValues(lengths, heads, kv, dim, F16, window=70, sinks=9, layout=layout, at=slice(0, 40))
        got = c.check_bwd(*c.check_fwd())
        assert all(bool(t.isfinite().all()) for t in got[:3])


def test_large_values_elsewhere():
    """A sequence's results are the same bits whatever another's values are."""
    plain = LargeValues([200, 200], 2, 1, 64, F16, at=slice(0, 0))
    o, lse = plain.fwd()
    want = plain.bwd(o, lse)
    c = LargeValues([200, 200], 2, 1, 64, F16, at=slice(0, 200))
    o2, lse2 = c.check_fwd()
    got = c.check_bwd(o2, lse2)
    assert torch.equal(o2[200:], o[200:]) and all(torch.equal(a[200:], b[200:]) for a, b in zip(got[:3], want[:3]))


def test_overflow_stays_an_overflow():
    """Gradients that do not fit binary16 are inf, and NaN goes in and comes out."""
    c = LargeValues([200], 1, 1, 64, F16)
    c.do = (c.do.double() * 1e6).to(F16)
    c.d["do"].copy_(c.do)
    o, lse = c.fwd()
    assert bool(c.bwd(o, lse)[0].isinf().any())
    c = Call([200], 1, 1, 64, F16)
    c.d["v"][7, 0, 3] = math.nan
    o, lse = c.fwd()
    assert bool(c.bwd(o, lse)[0].isnan().any())


class Far(Call):
    """One head: the first key takes all but exp(-gap) a key of every later query's weight.  q = a e0, k_0 = 32 e0, the other
    keys 8 e2; v_0 = 0, the other values 64 e1; do = g e1."""

    def __init__(self, n, dim, dtype, gap, g=1.0):
        super().__init__([n], 1, 1, dim, dtype, scale=0.125)
        for t in (self.q, self.k, self.v, self.do):
            t.zero_()
        self.gap = gap
        self.q[:, 0, 0] = gap / 4.0
        self.k[0, 0, 0] = 32.0
        self.k[1:, 0, 2] = 8.0
        self.v[1:, 0, 1] = 64.0
        self.do[:, 0, 1] = g
        for name in ("q", "k", "v", "do"):
            self.d[name].copy_(getattr(self, name))


N = 40000


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_many_small_weights(dtype, dim):
    """40000 keys of weight 2^-26: together 6e-4 of a row, 0.04 of its output, and each less than half of binary16's smallest
    number beside the largest weight."""
    c = Far(N, dim, dtype, 18.0)
    o, lse = c.fwd()
    i = torch.arange(N, dtype=torch.float64)
    w = i * math.exp(-18.0)
    want = torch.zeros(N, dim, dtype=torch.float64)
    want[:, 1] = 64.0 * w / (1.0 + w)
    # a weight and its row's sum: half a step of the weight; binary32's roundings of the score (gap 18: 8 u 18), its exponential
    # (8 u) and a sum of n terms (2 n u), and of the product's sum the same; binary16 below 2^-14 off by 2^-25, of weights in
    # units of 2^-7.  lse: the sum is 1 + w, of a lane's 32 terms of a tile first, then of its tiles: 2 (32 + n / 64 + 2) u of it
    e = want * (A.HALF[dtype] + (8 * 18 + 16 + 2 * 2 * N) * A.U)
    if dtype == F16:
        e[:, 1] += i * 2.0 ** -32 * 64.0
    close(o[:, 0], want, A.stored(e, want, dtype), "o")
    close(lse[0], 18.0 + torch.log1p(w), 18.0 * 8 * A.U + 2 * (34 + N / 64) * A.U + 16 * A.U + 0 * w, "lse")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_gradients_of_many_small_weights(dtype, dim):
    """Weights of 2^-31, each ds below binary16's smallest number in units of |do|."""
    g = 1024.0
    c = Far(N, dim, dtype, 21.5, g)
    o, lse = c.fwd()
    dq, dk, dv, _ = c.bwd(o, lse)
    i = torch.arange(N, dtype=torch.float64)
    p = torch.exp(-lse[0].cpu().double())                                # of every key but the first, whose score is 21.5
    delta = g * o[:, 0, 1].cpu().double()
    ds, ds0 = p * (64.0 * g - delta), -torch.exp(21.5 - lse[0].cpu().double()) * delta
    # binary32: the score and the difference (21.5, 8 u each) and the exponential, of ds; then half a step; binary16 2^-25 in
    # units of 2^-4 over twice |do|
    r = (8 * 2 * 21.5 + 16) * A.U + A.HALF[dtype]
    lost = 2.0 ** -25 * 2.0 ** -4 * 2.0 * g if dtype == F16 else 0.0
    depth = 2 * N * A.U
    want, e = (torch.zeros(N, dim, dtype=torch.float64) for _ in range(2))
    want[:, 0], want[:, 2] = 0.125 * 32.0 * ds0, 0.125 * 8.0 * i * ds
    e[:, 0] = 0.125 * 32.0 * (ds0.abs() * (r + depth) + lost)
    e[:, 2] = 0.125 * 8.0 * i * (ds * (r + depth) + lost)
    close(dq[:, 0], want, A.stored(e, want, dtype), "dq")
    after = lambda t: t.flip(0).cumsum(0).flip(0)                        # sums over the queries from the key on
    q0 = 21.5 / 4.0
    want, e = (torch.zeros(N, dim, dtype=torch.float64) for _ in range(2))
    want[:, 0] = 0.125 * q0 * after(ds)
    e[:, 0] = 0.125 * q0 * after(ds * (r + depth) + lost)
    want[0, 0] = 0.125 * q0 * ds0.sum()
    e[0, 0] = 0.125 * q0 * (ds0.abs() * (r + depth) + lost).sum()
    close(dk[:, 0], want, A.stored(e, want, dtype), "dk")
