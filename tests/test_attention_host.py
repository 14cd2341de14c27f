"""CPU tests of the attention operators: the 64-bit forms' gradients against
differences, the buckets' borders in whole numbers, and every refusal at the C
boundary and in the binding."""
import ctypes as C
import math
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

import attention_oracle as A

FAKE = 1 << 20          # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def Z():
    from zero_partitioned_mixed_flatten_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    import zero_partitioned_mixed_flatten_amd as Z
    return Z


# ---- the 64-bit forms ------------------------------------------------------------------

def _difference(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_gradient_against_differences(interleaved):
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, w, dy = n(5, 3, 12), n(12), n(5, 3, 12)
    cs = A.angles(range(5), 8, 100.0)
    (dx, dw), _ = A.qk_bwd(dy, x, w, cs, 1e-3, interleaved)
    for _ in range(3):
        d = n(5, 3, 12)
        assert math.isclose(float((dx * d).sum()), float(_difference(lambda v: (A.qk_fwd(v, w, cs, 1e-3, interleaved)[0] * dy).sum(), x, d)),
                            rel_tol=1e-6)
        d = n(12)
        assert math.isclose(float((dw * d).sum()), float(_difference(lambda v: (A.qk_fwd(x, v, cs, 1e-3, interleaved)[0] * dy).sum(), w, d)),
                            rel_tol=1e-6)


def test_the_turn_keeps_lengths_and_distances():
    """Turned by their positions, q and k meet in a product that goes by the distance alone."""
    g = torch.Generator().manual_seed(2)
    q, k = torch.randn(1, 1, 16, generator=g, dtype=torch.float64), torch.randn(1, 1, 16, generator=g, dtype=torch.float64)
    for interleaved in (False, True):
        at = lambda x, p: A.turned(x, A.angles([p], 16, 100.0), interleaved)
        a = (at(q, 9) * at(k, 4)).sum()
        assert torch.isclose(a, (at(q, 105) * at(k, 100)).sum(), rtol=1e-12)
        assert torch.isclose(at(q, 7).square().sum(), q.square().sum(), rtol=1e-12)
        assert torch.allclose(A.turned(at(q, 7), A.angles([7], 16, 100.0), interleaved, True), q, rtol=1e-12)


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 2), (1, 0), (5, 1)])
def test_attention_gradient_against_differences(window, sinks):
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    edges, hq, hk, d, starts = [0, 9, 9, 10, 17], 4, 2, 6, [0, 1, 3]
    q, k, v, bias, do = n(17, hq, d), n(17, hk, d), n(17, hk, d), n(hq, 3), n(17, hq, d)
    f = lambda q, k, v, b: A.attention_fwd(q, k, v, b, starts, 0.4, window, sinks, edges, torch.float32)[0]
    o, lse = f(q, k, v, bias)
    grads, _ = A.attention_bwd(do, o, lse, q, k, v, bias, starts, 0.4, window, sinks, edges, torch.float32)
    for i in range(4):
        args = [q, k, v, bias]
        dirn = n(*args[i].shape)
        want = _difference(lambda x: (f(*args[:i], x, *args[i + 1:])[0] * do).sum(), args[i], dirn)
        assert math.isclose(float((grads[i] * dirn).sum()), float(want), rel_tol=1e-6, abs_tol=1e-8)


def test_visible():
    see = A.visible(6, 2, 1)
    assert see.int().tolist() == [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0],
                                  [1, 0, 0, 0, 1, 1]]


# ---- buckets -------------------------------------------------------------------------------

@pytest.mark.parametrize("buckets,most", [(1, 7), (2, 2), (2, 100), (3, 50), (32, 128), (32, 256), (64, 33), (64, 4096), (64, 1 << 30), (7, 4)])
def test_borders(Z, buckets, most):
    """Each border is the first whole distance that reaches its ratio, or one past the bucket before."""
    starts = Z.zero_attention_buckets(buckets, most)
    half = buckets // 2
    n = buckets - half
    assert starts[0] == 0 and all(a < b for a, b in zip(starts, starts[1:]))
    assert starts[:half] == list(range(half))
    for b in range(n if buckets > 1 else 0):
        reaches = lambda d: Fraction(d, half) ** n >= Fraction(most, half) ** b
        d = starts[half + b]
        assert reaches(d) and (not reaches(d - 1) or d == starts[half + b - 1] + 1), (b, d)


def test_borders_refused(Z):
    L, E = Z.lib(), Z._lib
    out = (C.c_uint32 * 64)()
    assert L.zero_attention_buckets(None, 4, 10) == E.ZERO_EINVAL
    assert L.zero_attention_buckets(out, 0, 10) == E.ZERO_EINVAL
    assert L.zero_attention_buckets(out, 8, 4) == E.ZERO_EINVAL
    assert L.zero_attention_buckets(out, 65, 1000) == E.ZERO_ERANGE
    assert L.zero_attention_buckets(out, 8, (1 << 30) + 1) == E.ZERO_ERANGE


def test_params(Z):
    p = Z.attention_params(8, 2, 64, window=5, sinks=1, starts=[0, 4])
    assert (p.heads, p.kv_heads, p.dim, p.window, p.sinks, p.buckets, list(p.starts)[:3]) == (8, 2, 64, 5, 1, 2, [0, 4, 0])
    assert p.scale == 64 ** -0.5 and C.sizeof(p) == 296 == 16 + 8 + 8 + 8 + 4 * Z.ZERO_MAX_BUCKETS
    for bad in (dict(heads=-1), dict(window=-1), dict(sinks=1 << 32), dict(dim=0), dict(starts=range(65)), dict(starts=[-1])):
        with pytest.raises(ValueError):
            Z.attention_params(**{**dict(heads=8, kv_heads=2, dim=64), **bad})


# ---- the C boundary -----------------------------------------------------------------------------

def _fwd(Z, params=None, **kw):
    a = dict(o=FAKE, lse=FAKE, q=FAKE, k=FAKE, v=FAKE, ld=512, hs=64, bias=None, vec=Z.ZERO_F16, tokens=10, offsets=FAKE, n=2,
             dtype=Z.ZERO_F16)
    a.update(kw)
    p = Z.attention_params(8, 2, 64) if params is None else params
    h = lambda x: (a[x], a["ld"], a["hs"])
    return Z.lib().zero_attention_fwd(*h("o"), a["lse"], *h("q"), *h("k"), *h("v"), a["bias"], a["vec"], p, a["tokens"], a["offsets"],
                                      a["n"], a["dtype"], None)


def _bwd(Z, params=None, **kw):
    a = dict(dq=FAKE, dk=2 * FAKE, dv=3 * FAKE, dbias=None, grad=Z.ZERO_F16, do=FAKE, o=FAKE, lse=FAKE, q=FAKE, k=FAKE, v=FAKE, ld=512,
             hs=64, bias=None, vec=Z.ZERO_F16, tokens=10, offsets=FAKE, n=2, dtype=Z.ZERO_F16, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    p = Z.attention_params(8, 2, 64) if params is None else params
    h = lambda x: (a[x], a["ld"], a["hs"])
    return Z.lib().zero_attention_bwd(*h("dq"), *h("dk"), *h("dv"), a["dbias"], a["grad"], 0, *h("do"), *h("o"), a["lse"], *h("q"), *h("k"),
                                      *h("v"), a["bias"], a["vec"], p, a["tokens"], a["offsets"], a["n"], a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_attention_refusals(Z, call):
    E = Z._lib
    P = Z.attention_params
    nan, inf = math.nan, math.inf
    for p in (P(8, 3, 64), P(0, 1, 64), P(8, 0, 64), P(8, 2, 60), P(8, 2, 64, scale=0.0), P(8, 2, 64, scale=-1.0), P(8, 2, 64, scale=nan),
              P(8, 2, 64, scale=inf), P(8, 2, 64, scale=1e39), P(8, 2, 64, scale=1e-60), P(8, 2, 64, starts=[0, 1])):
        assert call(Z, p) == E.ZERO_EINVAL, (p.heads, p.kv_heads, p.dim, p.scale)
    for starts in ([1], [0, 0], [0, 5, 4]):
        assert call(Z, P(8, 2, 64, starts=starts), bias=FAKE) == E.ZERO_EINVAL, starts
    many = P(8, 2, 64, starts=[0])
    many.buckets = 65
    assert call(Z, many, bias=FAKE) == E.ZERO_ERANGE
    assert call(Z, P(8, 2, 136)) == E.ZERO_ERANGE
    assert call(Z, P((1 << 16) + 1, 1, 64)) == E.ZERO_ERANGE
    for bad in (dict(dtype=Z.ZERO_F32), dict(dtype=0), dict(bias=FAKE), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(n=0),
                dict(offsets=None, n=3)):
        assert call(Z, **bad) == E.ZERO_EINVAL, bad
    for bad in (dict(q=FAKE + 1), dict(offsets=FAKE + 2), dict(lse=FAKE + 2)):
        assert call(Z, **bad) == E.ZERO_EALIGN, bad
    assert call(Z, P(8, 2, 64, starts=[0]), bias=FAKE + 1) == E.ZERO_EALIGN
    assert call(Z, P(8, 2, 64, starts=[0]), bias=FAKE, vec=Z.ZERO_BF16) == E.ZERO_EINVAL
    for bad in (dict(ld=63), dict(hs=63), dict(ld=(1 << 50) + 1), dict(hs=(1 << 50) + 1), dict(ld=1 << 50, tokens=1 << 10, offsets=None, n=1),
                dict(tokens=(1 << 30) + 1), dict(n=(1 << 30) + 1), dict(n=1 << 29)):
        assert call(Z, **bad) == E.ZERO_ERANGE, bad
    empty = {n: None for n in ("o", "lse", "q", "k", "v", "dq", "dk", "dv", "do", "ws")}
    assert call(Z, tokens=0, n=0, offsets=None, **empty) == E.ZERO_OK
    assert call(Z, tokens=0, n=5, **empty) == E.ZERO_OK


def test_attention_null_params(Z):
    L = Z.lib()
    h = (FAKE, 512, 64)
    assert L.zero_attention_fwd(*h, FAKE, *h, *h, *h, None, 1, None, 1, None, 1, 1, None) == Z._lib.ZERO_EINVAL
    assert L.zero_attention_bwd(*h, *h, *h, None, 1, 0, *h, *h, FAKE, *h, *h, *h, None, 1, None, 1, None, 1, 1, FAKE, 1 << 20, None) == \
        Z._lib.ZERO_EINVAL
    assert L.zero_attention_workspace_bytes(None, 1, 1) == 0


def test_attention_backward_refusals(Z):
    E = Z._lib
    P = Z.attention_params
    for bad in (dict(dq=None), dict(dk=None), dict(dv=None), dict(do=None), dict(lse=None), dict(ws=None), dict(dk=FAKE), dict(dv=FAKE),
                dict(dv=2 * FAKE), dict(dbias=4 * FAKE)):
        assert _bwd(Z, **bad) == E.ZERO_EINVAL, bad
    assert _bwd(Z, ws=FAKE + 8) == E.ZERO_EALIGN
    need = Z.zero_attention_workspace_bytes(P(8, 2, 64), 10, 2)
    assert need >= 2 * 8 * 10 * 4 and _bwd(Z, wsb=need - 1) == E.ZERO_ERANGE
    b = P(8, 2, 64, starts=[0, 1])
    more = Z.zero_attention_workspace_bytes(b, 10, 2)
    assert more > need and _bwd(Z, b, bias=FAKE, dbias=4 * FAKE, wsb=more - 1) == E.ZERO_ERANGE
    assert _bwd(Z, b, bias=FAKE, dbias=4 * FAKE, grad=Z.ZERO_BF16) == E.ZERO_EINVAL
    assert _bwd(Z, b, bias=FAKE, dbias=4 * FAKE + 1) == E.ZERO_EALIGN
    assert Z.zero_attention_workspace_bytes(b, 0, 2) == Z.zero_attention_workspace_bytes(b, 10, 0) == 0


def _qk(Z, bwd, **kw):
    a = dict(qo=FAKE, ko=2 * FAKE, q=FAKE, k=FAKE, dqo=FAKE, dko=FAKE, wq=None, wk=None, vec=Z.ZERO_F16, ld=512, hs=64, tokens=10, hq=8, hk=2,
             dim=64, dtype=Z.ZERO_F16, eps=1e-6, table=FAKE, rows=10, rot=64, pos=None, dwq=4 * FAKE, dwk=5 * FAKE, grad=Z.ZERO_F16, ws=FAKE,
             wsb=1 << 30)
    a.update(kw)
    h = lambda x: (a[x], a["ld"], a["hs"])
    tail = (a["wq"], a["wk"], a["vec"], a["tokens"], a["hq"], a["hk"], a["dim"], a["dtype"], a["eps"], a["table"], a["rows"], a["rot"], 0,
            a["pos"], 0)
    if not bwd:
        return Z.lib().zero_qk_norm_rope_fwd(*h("qo"), *h("ko"), *h("q"), *h("k"), *tail, None)
    return Z.lib().zero_qk_norm_rope_bwd(*h("qo"), *h("ko"), a["dwq"], a["dwk"], a["grad"], 0, *h("dqo"), *h("dko"), *h("q"), *h("k"), *tail,
                                         a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_qk_refusals(Z, bwd):
    E = Z._lib
    for bad in (dict(qo=None), dict(q=None), dict(k=None), dict(ko=None), dict(ko=FAKE), dict(dtype=0), dict(dtype=4), dict(hq=0), dict(dim=0),
                dict(dim=63), dict(rot=63), dict(rot=66), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=1e39), dict(eps=1e-60),
                dict(table=None), dict(rows=0), dict(hk=0), dict(wq=FAKE, vec=Z.ZERO_BF16)):
        assert _qk(Z, bwd, **bad) == E.ZERO_EINVAL, bad
    for bad in (dict(q=FAKE + 1), dict(table=FAKE + 4), dict(pos=FAKE + 2), dict(wq=FAKE + 1), dict(wk=FAKE + 2, vec=Z.ZERO_F32)):
        assert _qk(Z, bwd, **bad) == E.ZERO_EALIGN, bad
    for bad in (dict(dim=258, ld=4096, hs=300), dict(tokens=(1 << 30) + 1), dict(hq=(1 << 16) + 1, ld=1 << 30), dict(ld=63), dict(hs=63),
                dict(rows=(1 << 30) + 1), dict(tokens=1 << 30, hq=1 << 16, ld=1 << 20), dict(ld=(1 << 50) + 1)):
        assert _qk(Z, bwd, **bad) == E.ZERO_ERANGE, bad
    nothing = dict(qo=None, ko=None, q=None, k=None, dqo=None, dko=None, tokens=0, dwq=None, dwk=None)
    assert _qk(Z, bwd, **nothing) == E.ZERO_OK


def test_qk_backward_refusals(Z):
    E = Z._lib
    for bad in (dict(dqo=None), dict(dko=None), dict(dwk=4 * FAKE), dict(ws=None), dict(grad=Z.ZERO_BF16),
                dict(hk=0, ko=None, k=None, dko=None)):
        assert _qk(Z, True, **bad) == E.ZERO_EINVAL, bad
    assert _qk(Z, True, ws=FAKE + 4) == E.ZERO_EALIGN
    assert _qk(Z, True, dwq=4 * FAKE + 1) == E.ZERO_EALIGN
    need = Z.zero_qk_workspace_bytes(10, 8, 2, 64)
    assert need > 0 and _qk(Z, True, wsb=need - 1) == E.ZERO_ERANGE


def test_rope_table_refusals(Z):
    L, E = Z.lib(), Z._lib
    for base in (0.0, -2.0, math.nan, math.inf):
        assert L.zero_rope_table(FAKE, 4, 64, base, None) == E.ZERO_EINVAL
    assert L.zero_rope_table(None, 4, 64, 10.0, None) == E.ZERO_EINVAL
    assert L.zero_rope_table(FAKE, 4, 63, 10.0, None) == E.ZERO_EINVAL
    assert L.zero_rope_table(FAKE + 8, 4, 64, 10.0, None) == E.ZERO_EALIGN
    assert L.zero_rope_table(FAKE, (1 << 30) + 1, 64, 10.0, None) == E.ZERO_ERANGE
    assert L.zero_rope_table(FAKE, 4, 258, 10.0, None) == E.ZERO_ERANGE
    assert L.zero_rope_table(None, 0, 64, 10.0, None) == E.ZERO_OK
    assert L.zero_rope_table(None, 4, 0, 10.0, None) == E.ZERO_OK


# ---- the binding ----------------------------------------------------------------------------------

class _Fake:
    """The face of a device tensor that need not be there."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.float16, device=0, strides=None):
        self.shape, self.dtype, self._device = torch.Size(shape), dtype, device
        self.device = f"cuda:{device}"
        n, s = 1, []
        for d in reversed(shape):
            s.append(n)
            n *= d
        self._strides, self._plain = tuple(strides or reversed(s)), strides is None

    def get_device(self):
        return self._device

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def stride(self):
        return self._strides

    def is_contiguous(self):
        return self._plain

    def data_ptr(self):
        return FAKE


class _Stream:
    cuda_stream = 0

    def __init__(self, device):
        self.device_index = device


@pytest.fixture
def bound(Z, monkeypatch):
    """The binding over a library that only counts its calls."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or (64 if name.endswith("bytes") else 0)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(Z._lib, "lib", lambda: Lib())
    monkeypatch.setattr(Z._lib, "_stream", lambda s: 0)
    return calls


def test_binding_attention(Z, bound):
    F, p = _Fake, Z.attention_params(4, 2, 64, starts=[0, 3])
    good = dict(o=F((10, 4, 64)), lse=F((4, 10), torch.float32), q=F((10, 4, 64)), k=F((10, 2, 64)), v=F((10, 2, 64)), params=p, bias=F((4, 2)),
                offsets=F((3,), torch.int32))
    Z.zero_attention_fwd(**good)
    Z.zero_attention_fwd(**{**good, "offsets": None, "sequences": 2, "stream": _Stream(0)})
    assert bound == ["zero_attention_fwd"] * 2
    bad = [dict(o=F((10, 4, 64), torch.float64)), dict(q=F((9, 4, 64))), dict(q=F((10, 2, 64))), dict(q=F((10, 4, 32))), dict(q=F((10, 256))),
           dict(k=F((10, 4, 64))), dict(v=F((10, 2, 64), torch.bfloat16)), dict(k=F((10, 2, 64), device=1)), dict(lse=F((4, 9), torch.float32)),
           dict(lse=F((4, 10))), dict(lse=F((10, 4), torch.float32)), dict(lse=F((4, 10), torch.float32, strides=(20, 1))),
           dict(q=F((10, 4, 64), strides=(1, 640, 10))), dict(bias=F((4, 3))), dict(bias=F((4, 2), torch.bfloat16)), dict(bias=F((8,))),
           dict(bias=F((4, 2), strides=(1, 4))), dict(offsets=F((3,), torch.int64)), dict(offsets=F((3, 1), torch.int32)),
           dict(offsets=F((0,), torch.int32)), dict(offsets=F((3,), torch.int32, device=1)), dict(offsets=F((3,), torch.int32, strides=(2,))),
           dict(offsets=None, sequences=-1), dict(stream=_Stream(1)), dict(o=F((10, 4, 64), device=1))]
    for b in bad:
        with pytest.raises((ValueError, TypeError)):
            Z.zero_attention_fwd(**{**good, **b})
    with pytest.raises(ValueError, match="device tensor"):
        Z.zero_attention_fwd(**{**good, "o": torch.zeros(10, 4, 64)})
    assert len(bound) == 2
    good = dict(dq=F((10, 4, 64)), dk=F((10, 2, 64)), dv=F((10, 2, 64)), dbias=F((4, 2), torch.float32), dout=F((10, 4, 64)), **good)
    Z.zero_attention_bwd(**{**good, "workspace": F((64,), torch.uint8)})
    assert bound[2:] == ["zero_attention_bwd"]
    for b in [dict(dq=F((10, 2, 64))), dict(dk=F((10, 4, 64))), dict(dv=F((11, 2, 64))), dict(dout=F((10, 4, 64), torch.float32)),
              dict(dbias=F((4, 3))), dict(workspace=F((64,), torch.uint8, device=1)), dict(workspace=F((64,), torch.uint8, strides=(2,)))]:
        with pytest.raises((ValueError, TypeError)):
            Z.zero_attention_bwd(**{"workspace": F((64,), torch.uint8), **good, **b})
    assert len(bound) == 3


def test_binding_qk(Z, bound):
    F = _Fake
    good = dict(q_out=F((10, 4, 64)), k_out=F((10, 2, 64)), q=F((10, 4, 64)), k=F((10, 2, 64)), wq=F((64,)), wk=F((64,)),
                table=F((100, 16, 2), torch.float32), positions=F((10,), torch.int32))
    Z.zero_qk_norm_rope_fwd(**good)
    Z.zero_qk_norm_rope_fwd(**{**good, "k": None, "k_out": None, "wk": None, "table": None})
    assert bound == ["zero_qk_norm_rope_fwd"] * 2
    bad = [dict(q_out=F((10, 256))), dict(q=F((10, 5, 64))), dict(k=None), dict(k_out=None), dict(k=F((9, 2, 64))), dict(wq=F((32,))),
           dict(wq=F((64,), torch.float32)), dict(wk=F((64,), torch.bfloat16)), dict(table=F((100, 16, 2))), dict(table=F((100, 32), torch.float32)),
           dict(table=F((100, 16, 2), torch.float32, strides=(64, 2, 1))), dict(positions=F((9,), torch.int32)),
           dict(positions=F((10,), torch.int64)), dict(k=F((10, 2, 64), strides=(1, 1, 2)))]
    for b in bad:
        with pytest.raises((ValueError, TypeError)):
            Z.zero_qk_norm_rope_fwd(**{**good, **b})
    assert len(bound) == 2
    del good["q_out"], good["k_out"]
    good.update(dq=F((10, 4, 64)), dk=F((10, 2, 64)), dwq=F((64,)), dwk=F((64,)), dq_out=F((10, 4, 64)), dk_out=F((10, 2, 64)),
                workspace=F((64,), torch.uint8))
    Z.zero_qk_norm_rope_bwd(**good)
    for b in [dict(dwq=F((64,), torch.float32)), dict(dwk=F((63,))), dict(dq_out=None), dict(dk=None), dict(dk_out=F((10, 4, 64)))]:
        with pytest.raises((ValueError, TypeError, AttributeError)):
            Z.zero_qk_norm_rope_bwd(**{**good, **b})
    assert len(bound) == 3
    Z.zero_rope_table(F((100, 16, 2), torch.float32))
    for t in (F((100, 32), torch.float32), F((100, 16, 2)), F((100, 16, 3), torch.float32)):
        with pytest.raises((ValueError, TypeError)):
            Z.zero_rope_table(t)
    assert len(bound) == 4


# ---- WindowAttention ------------------------------------------------------------------------------

def _place(Z, **kw):
    return Z.WindowAttention(16, 4, 2, 8, dtype=torch.float32, device="cpu", **kw)


def test_place_refusals(Z):
    q, k = torch.zeros(6, 4, 8), torch.zeros(6, 2, 8)
    for kw in (dict(bias=torch.zeros(4, 2)), dict(starts=[0])):
        with pytest.raises(ValueError, match="go together"):
            _place(Z, **kw)
    with pytest.raises(ValueError):
        Z.WindowAttention(-1, 4, 2, 8, device="cpu")
    with pytest.raises(ValueError):
        Z.WindowAttention(1, 4, 2, 8, max_sequences=0, device="cpu")
    p = _place(Z, table=torch.zeros(6, 4, 2))
    with pytest.raises(ValueError, match="made for"):
        p.forward(torch.zeros(17, 4, 8), torch.zeros(17, 2, 8), torch.zeros(17, 2, 8))
    with pytest.raises(ValueError, match="made for"):
        p.forward(q, k, k, sequences=2)
    with pytest.raises(ValueError, match="made for"):
        p.forward(q, k, k, offsets=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="positions"):
        p.forward(q, k, k, offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="no forward pass"):
        p.backward(q)
    with pytest.raises(ValueError, match="angles of 6"):
        p.forward(torch.zeros(7, 4, 8), torch.zeros(7, 2, 8), torch.zeros(7, 2, 8))
    p = Z.WindowAttention(16, 4, 2, 8, max_sequences=4, device="cpu")
    with pytest.raises(ValueError, match="equal length"):
        p.forward(q, k, k, sequences=4)
    with pytest.raises(ValueError, match="equal length"):
        p.forward(q, k, k, sequences=0)


def test_a_refused_forward_leaves_the_last_one(Z):
    """Refusals before anything is enqueued; one that comes later leaves no pass to go back over."""
    p = _place(Z)
    last = p._last = object()
    with pytest.raises(ValueError, match="made for"):
        p.forward(torch.zeros(17, 4, 8), torch.zeros(17, 2, 8), torch.zeros(17, 2, 8))
    assert p._last is last
    with pytest.raises(ValueError, match="device tensor"):
        p.forward(torch.zeros(6, 4, 8), torch.zeros(6, 2, 8), torch.zeros(6, 2, 8))
    assert p._last is None


def test_workspace_holds_smaller_batches(Z):
    """The workspace of a batch is enough for every smaller one: no more tokens in no more sequences."""
    rng = np.random.default_rng(5)
    for heads, kv, dim, window, sinks, buckets in [(64, 8, 128, 1024, 16, 0), (25, 25, 64, 0, 0, 32), (12, 3, 80, 700, 1, 24),
                                                   (1, 1, 8, 0, 0, 0), (8, 1, 128, 0, 0, 4), (600, 600, 64, 100, 200, 0)]:
        p = Z.attention_params(heads, kv, dim, window=window, sinks=sinks, starts=list(range(buckets)) or None)
        for most_tokens, most_n in [(8192, 1), (8192, 8), (20000, 3), (129, 2), (70, 70)]:
            whole = Z.zero_attention_workspace_bytes(p, most_tokens, most_n)
            assert whole > 0
            sizes = set(range(1, min(most_tokens, 300), 7)) | {int(t) for t in rng.integers(1, most_tokens + 1, 200)} | {most_tokens}
            for tokens in sizes:
                for n in range(1, most_n + 1):
                    assert Z.zero_attention_workspace_bytes(p, tokens, n) <= whole, (heads, kv, tokens, n)
        assert (Z.zero_qk_workspace_bytes(8192, heads, kv, dim) >=
                max(Z.zero_qk_workspace_bytes(t, heads, kv, dim) for t in range(1, 8193)))


def test_place_refuses_gradients_over_what_it_reads(Z):
    p = Z.WindowAttention(16, 4, 2, 8, device="cpu")
    q, k, v, o, do = (torch.zeros(7, h, 8, dtype=torch.float16) for h in (4, 2, 2, 4, 4))
    p._last = (q, k, v, q.clone(), k.clone(), o, None, {}, dict(offsets=None, sequences=1))
    for kw in (dict(dq=q), dict(dk=k), dict(dv=v), dict(dq=do), dict(dq=o)):
        with pytest.raises(ValueError, match="still read"):
            p.backward(do, **kw)
