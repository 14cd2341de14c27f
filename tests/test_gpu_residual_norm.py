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


def test_micro_batches_of_one_step_draw_their_own_masks():
    """A step accumulated over three micro-batches, the generator advanced
    after each backward pass: each drops its own elements, the same ones in
    both directions; two passes under one count would drop the same ones."""
    rows, cols, p = 40, 160, 0.5
    step = Z.AccumStep(cols, fused=False)
    step.init_state(1.0)
    rng = Z.LayerRng(77)
    place = Z.ResidualNorm(rows, cols, None, p=p, rng=rng, site=3)
    bias = torch.zeros(cols, device="cuda").half()
    biased = Z.ResidualNorm(rows, cols, None, bias=bias, p=p, rng=rng, site=4)
    x = torch.ones(rows, cols, device="cuda").half()
    g = torch.Generator()
    g.manual_seed(2)
    dy, dres = (torch.randn(rows, cols, generator=g).half().cuda() for _ in range(2))
    masks, total, bound = [], 0.0, 0.0
    for mb in range(3):
        print("[place] micro-batch", mb, flush=True)
        biased.forward(place.forward(x) * 0 + 1, place.r)
        dx, dr = biased.backward(dy, dres, grads=(None, None, step.grad32[:cols]), accumulate=mb > 0)
        place.backward(dx, dr)
        kept = (place.r != 0, biased.r != place.r)
        assert torch.equal(kept[1] & (dr != 0), dx != 0)          # the backward pass has the forward's mask
        masks.append(kept)
        total = total + dx.double().sum(0)
        # the sum takes dx before it is rounded to binary16 (half a step), in binary32 (rows + 32 roundings)
        bound = bound + dx.double().abs().sum(0) * (1.01 * 2.0 ** -11 + (rows + 32) * 2.0 ** -24) + rows * 2.0 ** -25
        rng.advance()
    torch.cuda.synchronize()
    assert rng.read().step == 3
    for k in range(2):
        for i in range(3):
            # half are kept, half of those agree between two draws: within five standard deviations
            assert abs(float(masks[i][k].double().mean()) - 0.5) < 5 * 0.5 / (rows * cols) ** 0.5
            agree = (masks[i][k] == masks[(i + 1) % 3][k]).double().mean()
            assert abs(float(agree) - 0.5) < 5 * 0.5 / (rows * cols) ** 0.5
    assert bool(((step.grad32[:cols].double() - total).abs() <= bound).all())
    place.forward(x)
    first = place.r.clone()
    place.forward(x)
    assert torch.equal(place.r, first)                            # no advance between: the same elements
