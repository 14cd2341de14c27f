"""Attention forward and backward on the GPU against the 64-bit forms, within
bounds derived from the roundings: types, head layouts, lengths from 0 and 1
across the tile edges, windows, first tokens, buckets, strides; sentinels round
every output."""
import itertools
import math

import pytest
import torch

import attention_oracle as A

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
SENTINEL = 123.0


def log(*a):
    print("[attention]", *a, flush=True)


def strided(tokens, heads, dim, dtype, layout, fill=SENTINEL):
    """A (tokens, heads, dim) view of a larger buffer: 'plain', 'joint' (a slice of wider rows), 'odd' (odd strides and
    an odd start), 'heads' (heads outermost)."""
    if layout == "plain":
        buf = torch.full((tokens, heads, dim), fill, dtype=dtype, device="cuda")
        return buf, buf
    if layout == "joint":
        buf = torch.full((tokens, heads * 3 * dim + 16), fill, dtype=dtype, device="cuda")
        return buf, buf[:, 8:8 + heads * 3 * dim].view(tokens, heads, 3 * dim)[:, :, dim:2 * dim]
    if layout == "odd":
        buf = torch.full((tokens * (heads * (dim + 3) + 5) + 7,), fill, dtype=dtype, device="cuda")
        return buf, torch.as_strided(buf, (tokens, heads, dim), (heads * (dim + 3) + 5, dim + 3, 1), 3)
    buf = torch.full((heads, tokens + 2, dim), fill, dtype=dtype, device="cuda")
    return buf, buf[:, 1:tokens + 1].transpose(0, 1)


def untouched(buf, view):
    """The buffer's elements outside the view still hold the sentinel."""
    keep = torch.ones_like(buf, dtype=torch.bool)
    offset = view.storage_offset() - buf.storage_offset()
    torch.as_strided(keep, view.shape, view.stride(), offset).fill_(False)
    return bool((buf[keep] == SENTINEL).all())


def normal(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * scale).to(dtype)


def close(got, want, bound, what):
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {i}: {float(got[i])} for {float(want[i])}, "
                             f"bound {float(bound[i]):.3g}; worst {float(((got - want).abs() / bound).nan_to_num(math.inf).max()):.3g}")


class Call:
    def __init__(self, lengths, heads, kv_heads, dim, dtype, window=0, sinks=0, starts=None, bias_dtype=None, layout="plain", after=0,
                 scale=None, equal=False, seed=0, spread=1.0, do_scale=1.0):
        g = torch.Generator().manual_seed(1000 + seed)
        self.edges = [0]
        for n in lengths:
            self.edges.append(self.edges[-1] + n)
        self.tokens, self.end = self.edges[-1] + after, self.edges[-1]
        self.dtype, self.starts, self.layout, self.window, self.sinks = dtype, starts, layout, window, sinks
        self.hq, self.hk, self.dim = heads, kv_heads, dim
        self.params = Z.attention_params(heads, kv_heads, dim, window, sinks, scale, starts)
        self.scale = self.params.scale
        T = self.tokens
        self.q, self.k, self.v = (normal(g, T, h, dim, dtype=dtype, scale=spread) for h in (heads, kv_heads, kv_heads))
        self.do = normal(g, T, heads, dim, dtype=dtype, scale=do_scale)
        self.bias = None if starts is None else normal(g, heads, len(starts), dtype=bias_dtype or dtype)
        offsets = torch.tensor(self.edges, dtype=torch.int32, device="cuda")
        self.where = {"sequences": len(lengths)} if equal else {"offsets": offsets}
        self.d = {n: self.device(getattr(self, n)) for n in ("q", "k", "v", "do")}
        self.dbias = None if self.bias is None else self.bias.cuda()

    def device(self, t):
        buf, view = strided(*t.shape, t.dtype, self.layout)
        view.copy_(t)
        return view

    def out(self, heads):
        return strided(self.tokens, heads, self.dim, self.dtype, self.layout)

    def f64(self, *names):
        return [getattr(self, n).double() for n in names]

    def fwd(self):
        buf, o = self.out(self.hq)
        lse = torch.full((self.hq, self.tokens), SENTINEL, device="cuda")
        Z.zero_attention_fwd(o, lse, self.d["q"], self.d["k"], self.d["v"], self.params, bias=self.dbias, **self.where)
        torch.cuda.synchronize()
        assert untouched(buf, o)
        return o, lse

    def want_fwd(self):
        return A.attention_fwd(*self.f64("q", "k", "v"), None if self.bias is None else self.bias.double(), self.starts, self.scale,
                               self.window, self.sinks, self.edges, self.dtype)

    def check_fwd(self):
        o, lse = self.fwd()
        n = self.end
        assert bool((o[n:] == SENTINEL).all()) and bool((lse[:, n:] == SENTINEL).all())
        (wo, wl), (eo, el) = self.want_fwd()
        close(lse[:, :n], wl[:, :n], el[:, :n] + A.stored(0 * el, wl, F32)[:, :n], "lse")
        close(o[:n], wo[:n], A.stored(eo, wo, self.dtype)[:n], "o")
        return o, lse

    def bwd(self, o, lse, grad_dtype=None, accumulate=False, start=0.0, workspace=None):
        outs = [self.out(h) for h in (self.hq, self.hk, self.hk)]
        db = None if self.bias is None else torch.full(self.bias.shape, start, dtype=grad_dtype or self.bias.dtype, device="cuda")
        Z.zero_attention_bwd(outs[0][1], outs[1][1], outs[2][1], db, self.d["do"], o, lse, self.d["q"], self.d["k"], self.d["v"], self.params,
                             bias=self.dbias, accumulate=accumulate, workspace=workspace, **self.where)
        torch.cuda.synchronize()
        for buf, view in outs:
            assert untouched(buf, view) and bool((view[self.end:] == SENTINEL).all())
        return [v for _, v in outs] + [db]

    def check_bwd(self, o, lse, grad_dtype=None, accumulate=False, start=0.0):
        got = self.bwd(o, lse, grad_dtype, accumulate, start)
        n = self.end
        cpu = lambda t: t.detach().cpu().double()
        oo, ll = cpu(o).masked_fill(torch.arange(self.tokens)[:, None, None] >= n, 0.0), cpu(lse)
        want, bound = A.attention_bwd(self.do.double(), oo, ll, *self.f64("q", "k", "v"), None if self.bias is None else self.bias.double(),
                                      self.starts, self.scale, self.window, self.sinks, self.edges, self.dtype)
        for name, x, w, e in zip(("dq", "dk", "dv"), got, want, bound):
            close(x[:n], w[:n], A.stored(e, w, self.dtype)[:n], name)
        if got[3] is not None:
            w = want[3] + (start if accumulate else 0.0)
            close(got[3], w, A.stored(bound[3] + 2 * A.U * w.abs(), w, got[3].dtype), "dbias")
        return got


LENGTHS = [[1], [2, 0, 1, 5], [31, 33, 64], [63, 65], [127, 1, 129], [128, 128], [300], [200, 0, 0, 333, 1, 77]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_lengths(lengths, dtype):
    for dim in (64, 128):
        log("lengths", lengths, dtype, dim)
        c = Call(lengths, 3, 3, dim, dtype, after=3)
        c.check_bwd(*c.check_fwd())


MASKS = [(1, 0), (2, 1), (31, 0), (64, 4), (65, 64), (100, 65), (128, 3), (200, 129), (7, 500), (299, 1), (300, 4), (1 << 40, 2)]


@pytest.mark.parametrize("window,sinks", MASKS)
def test_masks(window, sinks):
    for lengths, dtype, dim in (([300], F16, 64), ([130, 1, 259, 300], BF16, 128)):
        log("masks", window, sinks, lengths)
        c = Call(lengths, 2, 2, dim, dtype, window=window, sinks=sinks)
        c.check_bwd(*c.check_fwd())


@pytest.mark.parametrize("dim", [8, 16, 24, 32, 40, 56, 64, 72, 80, 96, 104, 112, 120, 128])
def test_dims(dim):
    for dtype in (F16, BF16):
        log("dim", dim, dtype)
        c = Call([70, 131], 2, 1, dim, dtype, window=90, sinks=2)
        c.check_bwd(*c.check_fwd())


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 2), (8, 1), (6, 2), (25, 25), (12, 3)])
def test_heads(heads, kv_heads):
    log("heads", heads, kv_heads)
    c = Call([140, 65], heads, kv_heads, 64, BF16, window=70, sinks=3)
    c.check_bwd(*c.check_fwd())


STARTS = {"one": [0], "two": [0, 1], "logs": Z.zero_attention_buckets(32, 128), "wide": Z.zero_attention_buckets(64, 4000),
          "steps": [0, 5, 64, 65, 100, 128, 129, 250], "far": [0, 1000]}


@pytest.mark.parametrize("starts", STARTS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
def test_bias(starts, window, sinks):
    for dtype, dim, bias_dtype in ((F16, 64, F16), (BF16, 128, F32), (BF16, 64, BF16)):
        log("bias", starts, window, sinks, dtype, dim)
        c = Call([300, 1, 129], 4, 2, dim, dtype, window, sinks, STARTS[starts], bias_dtype, after=1)
        c.check_bwd(*c.check_fwd())


@pytest.mark.parametrize("layout", ["joint", "odd", "heads"])
def test_layouts(layout):
    for dim, starts in ((64, None), (80, STARTS["logs"]), (128, None)):
        log("layout", layout, dim)
        c = Call([100, 70], 4, 2, dim, F16, window=60, sinks=2, starts=starts, layout=layout, after=2)
        c.check_bwd(*c.check_fwd())


def test_equal_lengths():
    for n, seqs in ((1, 5), (64, 3), (129, 4)):
        log("equal", n, seqs)
        c = Call([n] * seqs, 2, 2, 64, F16, equal=True)
        c.check_bwd(*c.check_fwd())


def test_many_sequences():
    """More sequences than lanes of a wave, many of them empty."""
    lengths = [(7 * i) % 11 if i % 3 else 0 for i in range(200)]
    c = Call(lengths, 2, 1, 64, BF16, window=5, sinks=1, starts=STARTS["two"], after=4)
    c.check_bwd(*c.check_fwd())


@pytest.mark.parametrize("grad_dtype,accumulate", [(F16, False), (F32, False), (F16, True), (F32, True)])
def test_bias_gradient_types(grad_dtype, accumulate):
    c = Call([200, 50], 3, 3, 64, F16, starts=STARTS["logs"], bias_dtype=F32)
    c.check_bwd(*c.check_fwd(), grad_dtype=grad_dtype, accumulate=accumulate, start=3.5)


@pytest.mark.parametrize("do_scale", [1e-6, 1e-3, 300.0])
def test_gradient_scale(do_scale):
    """Gradients far from 1: binary16's few exponents are used from where they are."""
    for dtype in (F16, BF16):
        log("scale", do_scale, dtype)
        c = Call([333], 2, 1, 64, dtype, window=100, sinks=2, do_scale=do_scale)
        c.check_bwd(*c.check_fwd())


@pytest.mark.parametrize("sinks", [1, 33, 128, 129])
def test_long_sequences_with_first_tokens(sinks):
    """The queries behind the window, a thousand at a time, on the keys of the first tokens."""
    for lengths, heads, kv_heads, dtype, dim in (([2500], 2, 1, F16, 64), ([1100, 40, 2100], 2, 2, BF16, 128)):
        log("long", sinks, lengths)
        c = Call(lengths, heads, kv_heads, dim, dtype, window=70, sinks=sinks, after=5)
        c.check_bwd(*c.check_fwd())


def test_long_sequence_with_bias():
    c = Call([2200], 4, 1, 64, F16, window=600, sinks=9, starts=Z.zero_attention_buckets(32, 1000))
    c.check_bwd(*c.check_fwd())
    c = Call([1700], 8, 1, 128, BF16, starts=Z.zero_attention_buckets(16, 300), bias_dtype=F32)
    c.check_bwd(*c.check_fwd())
