"""ResidualNorm on the GPU: what a refused call leaves behind, and how it is
used over several micro-batches."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402


def test_backward_after_a_refused_forward():
    """A forward pass that is refused changes nothing: backward is still the
    one of the last forward pass that ran."""
    g = torch.Generator()
    g.manual_seed(1)
    draw = lambda rows: torch.randn(rows, 64, generator=g).half().cuda()
    w = draw(1)[0]
    place, same = (Z.ResidualNorm(16, 64, w) for _ in range(2))
    x, dy = draw(5), draw(5)
    print("[place] refused forward", flush=True)
    for p in (place, same):
        p.forward(x)
    for bad in (draw(9).float(), draw(9).cpu(), torch.zeros(17, 64, device="cuda").half()):
        with pytest.raises((TypeError, ValueError)):
            place.forward(bad)
    assert place.rows == 5 and torch.equal(place.r, x)
    got, want = place.backward(dy), same.backward(dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(place.dw, same.dw)
