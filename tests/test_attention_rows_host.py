"""Refusals of the call that clears the rows in no sequence."""
import pytest
import torch

from test_attention_host import FAKE, Z, _Fake, bound  # noqa: F401  (fixtures)


def test_refusals(Z):  # noqa: F811
    E = Z._lib

    def call(**kw):
        a = dict(x=FAKE, ld=512, hs=64, tokens=10, heads=8, dim=64, dtype=Z.ZERO_F16, offsets=FAKE, n=2)
        a.update(kw)
        return Z.lib().zero_attention_clear_rows(a["x"], a["ld"], a["hs"], a["tokens"], a["heads"], a["dim"], a["dtype"], a["offsets"], a["n"],
                                                 None)

    for bad in (dict(x=None), dict(dtype=0), dict(dtype=4), dict(heads=0), dict(dim=0), dict(dim=60), dict(offsets=None)):
        assert call(**bad) == E.ZERO_EINVAL, bad
    for bad in (dict(x=FAKE + 1), dict(x=FAKE + 2, dtype=Z.ZERO_F32), dict(offsets=FAKE + 2)):
        assert call(**bad) == E.ZERO_EALIGN, bad
    for bad in (dict(dim=136), dict(heads=(1 << 16), ld=1 << 30), dict(tokens=(1 << 30) + 1), dict(n=(1 << 30) + 1), dict(ld=63), dict(hs=63),
                dict(ld=(1 << 50) + 1), dict(hs=(1 << 50) + 1)):
        assert call(**bad) == E.ZERO_ERANGE, bad
    assert call(x=None, tokens=0) == E.ZERO_OK


def test_binding(Z, bound):  # noqa: F811
    F = _Fake
    Z.zero_attention_clear_rows(F((10, 4, 64)), F((3,), torch.int32))
    assert bound == ["zero_attention_clear_rows"]
    for x, offsets in ((F((10, 256)), F((3,), torch.int32)), (F((10, 4, 64), torch.float64), F((3,), torch.int32)),
                       (F((10, 4, 64)), None), (F((10, 4, 64)), F((3,), torch.int64)), (F((10, 4, 64)), F((0,), torch.int32)),
                       (F((10, 4, 64)), F((3,), torch.int32, device=1)), (F((10, 4, 64), device=1), F((3,), torch.int32)),
                       (F((10, 4, 64), strides=(1, 640, 10)), F((3,), torch.int32))):
        with pytest.raises((ValueError, TypeError)):
            Z.zero_attention_clear_rows(x, offsets)
    assert len(bound) == 1
