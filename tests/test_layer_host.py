"""CPU checks of the layer operators: the 64-bit forms the GPU tests compare
with are pinned (published vectors of the generator, differences for the
gradients), and every argument error is reported before any device work."""
import ctypes as C

import numpy as np
import pytest

import layer_oracle as O

FAKE = 1 << 20          # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def Z():
    import os

    from zero_partitioned_mixed_flatten_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    import zero_partitioned_mixed_flatten_amd as Z
    return Z


# ---- the 64-bit forms ---------------------------------------------------------------

@pytest.mark.parametrize("counter,key,want", [
    # the generator's published known-answer vectors (Philox4x32, 10 rounds)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_generator_known_answers(counter, key, want):
    assert tuple(int(v) for v in O.philox4x32(counter, key)) == want


def test_mask_words_and_rate():
    k = O.keep(64, 1601, 0.1, seed=(5 << 40) | 77, step=3, site=9)
    # one element by hand: row 2, column 1600 is word 0 of the row's last group
    g = 2 * 201 + 200
    word = int(O.philox4x32((g, 0, 9, 3), (((5 << 40) | 77) & 0xFFFFFFFF, 5 << 8))[0]) & 0xFFFF
    assert k[2, 1600] == (word >= 6554)
    n = k.size
    assert abs(k.mean() - (1 - 6554 / 65536)) < 5 * np.sqrt(0.1 * 0.9 / n)      # five standard deviations
    assert O.threshold(0.0) == 0 and O.threshold(1.0) == 65536 and O.scale(1.0) == 0.0
    assert not O.keep(3, 5, 1.0, 1, 0, 0).any() and O.keep(3, 5, 0.0, 1, 0, 0).all()
    # other sites, steps, seeds: other masks
    base = O.keep(8, 64, 0.5, 1, 0, 0)
    for other in (O.keep(8, 64, 0.5, 2, 0, 0), O.keep(8, 64, 0.5, 1, 1, 0), O.keep(8, 64, 0.5, 1, 0, 1),
                  O.keep(8, 64, 0.5, 1 << 32 | 1, 0, 0)):
        assert 0.3 < (other == base).mean() < 0.7


def test_backward_forms_match_differences():
    """The backward formulas against central differences of the forward ones
    in 64 bits: a step of 1e-5 leaves a truncation error of order 1e-10 and a
    rounding error of order 1e-11."""
    rng = np.random.default_rng(3)
    rows, n, eps = 4, 11, 1e-3
    x, res, c, cr = (rng.standard_normal((rows, n)) for _ in range(4))
    w, b, bias = (rng.standard_normal(n) for _ in range(3))
    kept, s = O.keep(rows, n, 0.3, 9, 1, 2), O.scale(0.3)

    def loss(x, res, w, b, bias):
        r = res + O.dropped(x + bias, kept, s)
        y = O.norm_fwd(r, w, b, eps, "f32")[0][0]
        return float((y * c).sum() + (r * cr).sum())

    r = res + O.dropped(x + bias, kept, s)
    (y, mean, rstd), _ = O.norm_fwd(r, w, b, eps, "f32")
    (e, dw, db), _ = O.norm_bwd(c, r, mean, rstd, w, cr)
    dx = O.dropped(e, kept, s)
    for arg, grad in ((0, dx), (1, e), (2, dw), (3, db), (4, dx.sum(0))):
        base = [x, res, w, b, bias]
        num = np.empty_like(base[arg])
        for i in np.ndindex(num.shape):
            v = []
            for h in (1e-5, -1e-5):
                t = [a.copy() for a in base]
                t[arg][i] += h
                v.append(loss(*t))
            num[i] = (v[0] - v[1]) / 2e-5
        assert np.abs(num - grad).max() < 1e-7, arg


# ---- refusals: every case returns before any device work ---------------------------------

def _call(Z, fn, **kw):
    """One entry point with acceptable arguments, except those in kw."""
    names = {
        "zero_dropout_fwd": "out ld_out x ld_x residual ld_residual vec vec_dtype rows cols dtype p rng site stream",
        "zero_dropout_bwd": "dx ld_dx dbias grad_dtype accumulate dy ld_dy rows cols dtype p rng site ws ws_bytes stream",
        "zero_layernorm_fwd": "y ld_y mean rstd x ld_x w b vec_dtype rows cols dtype eps stream",
        "zero_layernorm_bwd": "dx ld_dx dw db grad_dtype accumulate dy ld_dy dres ld_dres x ld_x mean rstd w vec_dtype "
                              "rows cols dtype ws ws_bytes stream",
        "zero_dropout_layernorm_fwd": "r ld_r y ld_y mean rstd x ld_x residual ld_residual bias w b vec_dtype rows cols "
                                      "dtype eps p rng site stream",
        "zero_dropout_layernorm_bwd": "dx ld_dx dr ld_dr dw db dbias grad_dtype accumulate dy ld_dy dres ld_dres r ld_r "
                                      "mean rstd w vec_dtype rows cols dtype p rng site ws ws_bytes stream"}[fn].split()
    a = dict(vec_dtype=Z.ZERO_F32, grad_dtype=Z.ZERO_F32, accumulate=0, rows=4, cols=64, dtype=Z.ZERO_F16, p=0.1,
             site=0, eps=1e-5, ws_bytes=1 << 30, stream=None)
    out = []
    for i, n in enumerate(names):
        if n in kw:
            out.append(kw[n])
        elif n in a:
            out.append(a[n])
        elif n.startswith("ld_"):
            out.append(64)
        else:
            out.append(FAKE + 4096 * i)
    assert set(kw) <= set(names), (fn, kw)
    return getattr(Z.lib(), fn)(*out)


ALL = ["zero_dropout_fwd", "zero_dropout_bwd", "zero_layernorm_fwd", "zero_layernorm_bwd", "zero_dropout_layernorm_fwd",
       "zero_dropout_layernorm_bwd"]
MATRICES = {"zero_dropout_fwd": ["out", "x"], "zero_dropout_bwd": ["dx", "dy"], "zero_layernorm_fwd": ["y", "x"],
            "zero_layernorm_bwd": ["dx", "dy", "x"], "zero_dropout_layernorm_fwd": ["r", "y", "x"],
            "zero_dropout_layernorm_bwd": ["dx", "dr", "dy", "r"]}
OPTIONAL = {"zero_dropout_fwd": ["residual"], "zero_layernorm_bwd": ["dres"],
            "zero_dropout_layernorm_fwd": ["residual"], "zero_dropout_layernorm_bwd": ["dres"]}
VECTORS = {"zero_dropout_fwd": [("vec", "vec_dtype")], "zero_dropout_bwd": [("dbias", "grad_dtype")],
           "zero_layernorm_fwd": [("w", "vec_dtype"), ("b", "vec_dtype")],
           "zero_layernorm_bwd": [("dw", "grad_dtype"), ("db", "grad_dtype"), ("w", "vec_dtype")],
           "zero_dropout_layernorm_fwd": [("bias", "vec_dtype"), ("w", "vec_dtype"), ("b", "vec_dtype")],
           "zero_dropout_layernorm_bwd": [("dw", "grad_dtype"), ("db", "grad_dtype"), ("dbias", "grad_dtype"),
                                          ("w", "vec_dtype")]}


@pytest.mark.parametrize("fn", ALL)
def test_matrices_are_checked(Z, fn):
    E = Z._lib
    for m in MATRICES[fn]:
        assert _call(Z, fn, **{m: None}) == E.ZERO_EINVAL, m
    for m in MATRICES[fn] + OPTIONAL.get(fn, []):
        assert _call(Z, fn, **{m: FAKE + 1}) == E.ZERO_EALIGN, m
        assert _call(Z, fn, dtype=E.ZERO_F32, **{m: FAKE + 2}) == E.ZERO_EALIGN, m
        assert _call(Z, fn, **{"ld_" + m: 63}) == E.ZERO_ERANGE, m
        assert _call(Z, fn, **{"ld_" + m: 0}) == E.ZERO_ERANGE, m
        assert _call(Z, fn, **{"ld_" + m: 1 << 55}) == E.ZERO_ERANGE, m
        assert _call(Z, fn, **{"ld_" + m: (1 << 64) - 1}) == E.ZERO_ERANGE, m
    for dtype in (0, 4, -1):
        assert _call(Z, fn, dtype=dtype) == E.ZERO_EINVAL
    assert _call(Z, fn, rows=(1 << 40) + 1) == E.ZERO_ERANGE
    assert _call(Z, fn, cols=(1 << 30) + 1) == E.ZERO_ERANGE


@pytest.mark.parametrize("fn", ALL)
def test_vectors_are_checked(Z, fn):
    E = Z._lib
    for v, t in VECTORS[fn]:
        assert _call(Z, fn, **{v: FAKE + 2}) == E.ZERO_EALIGN, v
        assert _call(Z, fn, **{v: FAKE + 1, t: E.ZERO_F16}) == E.ZERO_EALIGN, v
        assert _call(Z, fn, **{t: E.ZERO_BF16}) == E.ZERO_EINVAL, v          # matrices are fp16 here
        assert _call(Z, fn, **{t: 7}) == E.ZERO_EINVAL, v


@pytest.mark.parametrize("fn", [f for f in ALL if "dropout" in f])
def test_dropout_arguments_are_checked(Z, fn):
    E = Z._lib
    for p in (-0.1, 1.5, float("nan"), float("inf")):
        assert _call(Z, fn, p=p) == E.ZERO_EINVAL
    assert _call(Z, fn, rng=None) == E.ZERO_EINVAL
    assert _call(Z, fn, rng=FAKE + 4) == E.ZERO_EALIGN


@pytest.mark.parametrize("fn", ["zero_layernorm_fwd", "zero_dropout_layernorm_fwd"])
def test_norm_forward_arguments_are_checked(Z, fn):
    E = Z._lib
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-60):
        assert _call(Z, fn, eps=eps) == E.ZERO_EINVAL
    assert _call(Z, fn, cols=0) == E.ZERO_ERANGE
    assert _call(Z, fn, mean=FAKE + 2) == E.ZERO_EALIGN
    assert _call(Z, fn, rstd=FAKE + 1) == E.ZERO_EALIGN
    if fn == "zero_dropout_layernorm_fwd":
        assert _call(Z, fn, r=FAKE, y=FAKE) == E.ZERO_EINVAL
    assert _call(Z, fn, mean=FAKE, rstd=FAKE) == E.ZERO_EINVAL
    assert _call(Z, fn, rows=0) == E.ZERO_OK                               # nothing to do


@pytest.mark.parametrize("fn", ["zero_layernorm_bwd", "zero_dropout_layernorm_bwd"])
def test_norm_backward_arguments_are_checked(Z, fn):
    E = Z._lib
    need = Z.zero_layer_workspace_bytes(4, 64)
    assert need > 0
    assert _call(Z, fn, ws_bytes=need - 1) == E.ZERO_ERANGE
    assert _call(Z, fn, ws=None) == E.ZERO_EINVAL
    assert _call(Z, fn, ws=FAKE + 8) == E.ZERO_EALIGN
    assert _call(Z, fn, mean=None) == E.ZERO_EINVAL and _call(Z, fn, rstd=None) == E.ZERO_EINVAL
    assert _call(Z, fn, mean=FAKE + 2) == E.ZERO_EALIGN and _call(Z, fn, rstd=FAKE + 2) == E.ZERO_EALIGN
    assert _call(Z, fn, cols=0) == E.ZERO_ERANGE
    assert _call(Z, fn, dw=FAKE, db=FAKE) == E.ZERO_EINVAL
    if fn == "zero_dropout_layernorm_bwd":
        assert _call(Z, fn, dx=FAKE, dr=FAKE) == E.ZERO_EINVAL
        assert _call(Z, fn, dbias=FAKE, db=FAKE) == E.ZERO_EINVAL
        assert _call(Z, fn, dbias=FAKE, dw=FAKE) == E.ZERO_EINVAL
    # no rows and no gradient wanted: nothing to do
    none = dict(dw=None, db=None, rows=0, dx=None, dy=None)
    if fn == "zero_dropout_layernorm_bwd":
        none.update(dbias=None, dr=None, r=None)
    assert _call(Z, fn, **none) == E.ZERO_OK


def test_dropout_empty_and_workspace(Z):
    E = Z._lib
    assert _call(Z, "zero_dropout_fwd", rows=0) == E.ZERO_OK
    assert _call(Z, "zero_dropout_fwd", cols=0) == E.ZERO_OK
    assert _call(Z, "zero_dropout_bwd", cols=0) == E.ZERO_OK
    assert _call(Z, "zero_dropout_bwd", rows=0, dbias=None) == E.ZERO_OK
    assert _call(Z, "zero_dropout_bwd", ws=None) == E.ZERO_EINVAL
    assert _call(Z, "zero_dropout_bwd", ws_bytes=Z.zero_layer_workspace_bytes(4, 64) - 1) == E.ZERO_ERANGE
    assert _call(Z, "zero_dropout_bwd", ws=FAKE + 4) == E.ZERO_EALIGN


def test_generator_arguments_are_checked(Z):
    E, L = Z._lib, Z.lib()
    assert L.zero_rng_init(None, 1, None) == E.ZERO_EINVAL and L.zero_rng_init(FAKE + 4, 1, None) == E.ZERO_EALIGN
    assert L.zero_rng_advance(None, None) == E.ZERO_EINVAL and L.zero_rng_advance(FAKE + 4, None) == E.ZERO_EALIGN
    assert C.sizeof(Z.RngState) == Z.RNG_BYTES == 16


def test_workspace_size(Z):
    W = Z.zero_layer_workspace_bytes
    assert W(0, 64) == 0 and W(64, 0) == 0 and W((1 << 40) + 1, 8) == 0 and W(8, (1 << 30) + 1) == 0
    for rows, cols in ((1, 1), (1, 8192), (7, 1601), (16384, 8192), (1 << 20, 64), (1 << 40, 1)):
        assert W(rows, cols) == W(rows, cols) > 0
    last = 0
    for rows in [*range(1, 3000), *range(3000, 70_000, 97)]:        # never less for more rows
        assert W(rows, 1600) >= last
        last = W(rows, 1600)
    # at the largest sizes it stays a small part of the matrices' own bytes
    assert W(16384, 8192) < 16384 * 8192 * 2


def test_flatten_still_refuses_bf16(Z):
    arr, k = Z.make_segments([(FAKE, 0, 0, 100)])
    assert Z.lib().zero_flatten_bucket(arr, k, FAKE, 100, Z.ZERO_BF16, 0, None) == Z._lib.ZERO_EINVAL


# ---- the binding's own checks ----------------------------------------------------------------

def test_binding_refuses_host_tensors(Z):
    import torch
    x = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        Z.zero_dropout_fwd(x, x, 0.1, None)
    with pytest.raises(ValueError, match="device tensor"):
        Z.zero_layernorm_fwd(x, None, None, x, None, None)


class _Fake:
    """A tensor's face, on a device that is not there."""

    def __init__(self, device, shape=(4, 64), dtype=None, stride=None):
        import torch
        self.shape, self.dtype, self._d = shape, dtype or torch.float16, device
        self.is_cuda, self._s = True, stride or (shape[-1], 1)
        self.device = f"cuda:{device}"

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def get_device(self):
        return self._d

    def is_contiguous(self):
        return self._s == (self.shape[-1], 1)

    def stride(self, i):
        return self._s[i]

    def data_ptr(self):
        return FAKE


def test_binding_refuses_other_devices_types_and_shapes(Z, monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(Z._lib, "_stream", lambda s: 0)

    def call(out=None, x=None, stream=None, **kw):
        Z.zero_dropout_fwd(out or _Fake(0), x or _Fake(0), 0.0, None, stream=stream, **kw)

    class S:
        device_index, cuda_stream = 1, 0

    with pytest.raises(ValueError, match="current device"):
        call(out=_Fake(1), x=_Fake(1))
    with pytest.raises(ValueError, match="stream belongs"):
        call(stream=S())
    for bad in (_Fake(1), _Fake(0, dtype=torch.float32)):
        with pytest.raises(TypeError):
            call(x=bad)
    for bad in (_Fake(0, (4, 63)), _Fake(0, (3, 64)), _Fake(0, (4, 64), stride=(1, 4)),
                _Fake(0, (2, 2, 64), stride=(256, 64, 1))):
        with pytest.raises(ValueError):
            call(x=bad)
    with pytest.raises(TypeError):
        call(out=_Fake(0, dtype=torch.float64))
    with pytest.raises(TypeError):
        call(bias=_Fake(0, (64,), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        call(bias=_Fake(0, (63,), stride=(63, 1)))
    with pytest.raises(ValueError):
        call(bias=_Fake(1, (64,), stride=(64, 1)))
    with pytest.raises(Z.ZeroError):                                # a broadcast row: the library refuses ld < cols
        call(x=_Fake(0, (4, 64), stride=(0, 1)))
    for site in (-1, 1 << 32):
        with pytest.raises(ValueError, match="site"):
            Z.zero_dropout_fwd(_Fake(0), _Fake(0), 0.0, None, site=site)
    for seed in (-1, 1 << 64):
        with pytest.raises(ValueError, match="seed"):
            Z.zero_rng_init(FAKE, seed)
    with pytest.raises(TypeError, match="share one type"):
        Z.zero_layernorm_fwd(_Fake(0), None, None, _Fake(0), _Fake(0, (64,), stride=(64, 1)),
                             _Fake(0, (64,), dtype=torch.float32, stride=(64, 1)))
    with pytest.raises(ValueError, match="one per row"):
        Z.zero_layernorm_fwd(_Fake(0), _Fake(0, (3,), dtype=torch.float32, stride=(3, 1)), None, _Fake(0), None, None)


@pytest.mark.parametrize("max_rows,cols", [(-1, 8), (4, 0), (4, -8)])
def test_residual_norm_refuses_shapes_without_columns(Z, max_rows, cols):
    with pytest.raises(ValueError, match="ResidualNorm"):
        Z.ResidualNorm(max_rows, cols, None)
