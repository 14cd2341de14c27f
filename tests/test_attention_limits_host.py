"""Batches with more workgroups than a launch holds are refused before anything
is enqueued, as the header says."""
import pytest

from test_attention_host import FAKE, Z, _bwd, _fwd  # noqa: F401  (fixture and calls)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_more_pieces_than_a_launch_holds(Z, call):  # noqa: F811
    E, P = Z._lib, Z.attention_params
    wide = dict(ld=25 * 64, tokens=700000, wsb=1 << 60)
    if call is _fwd:
        del wide["wsb"]
    for kw in (dict(offsets=FAKE, n=700000), dict(offsets=None, n=700000), dict(offsets=FAKE, n=671078)):
        assert call(Z, P(25, 25, 64), **{**wide, **kw}) == E.ZERO_ERANGE, kw
    assert Z.zero_attention_workspace_bytes(P(25, 25, 64), 700000, 700000) == 0
    # of equal lengths, not with offsets
    assert Z.zero_attention_workspace_bytes(P(25, 25, 64), 668000, 668000) > 0
    assert call(Z, P(25, 25, 64), **{**wide, "tokens": 668000, "n": 668000}) == E.ZERO_ERANGE


def test_more_queries_behind_the_window_than_a_launch_holds(Z):  # noqa: F811
    E, P = Z._lib, Z.attention_params
    p = P(1, 1, 8, window=1, sinks=1)
    assert _bwd(Z, p, ld=8, hs=8, tokens=1 << 30, n=1 << 22, offsets=None, wsb=1 << 60) == E.ZERO_ERANGE
    p = P(1, 1, 8, window=1, sinks=1)
    assert _bwd(Z, p, ld=8, hs=8, tokens=1 << 30, n=1 << 22, offsets=FAKE, wsb=1 << 60) == E.ZERO_ERANGE
