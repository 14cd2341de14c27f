"""CPU checks of what the layer operators and ResidualNorm refuse, and of what
a refused call leaves behind."""
import pytest

FAKE = 1 << 20          # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def Z():
    import os

    from zero_partitioned_mixed_flatten_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    import zero_partitioned_mixed_flatten_amd as Z
    return Z


# ---- eps -------------------------------------------------------------------------------

def _norm_fwd(Z, eps):
    """A layer norm of no rows: the arguments are checked, nothing is enqueued."""
    return Z.lib().zero_layernorm_fwd(None, 0, None, None, None, 0, None, None, Z.ZERO_F32, 0, 64, Z.ZERO_F16, eps, None)


def _joined_fwd(Z, eps):
    return Z.lib().zero_dropout_layernorm_fwd(None, 0, None, 0, None, None, None, 0, None, 0, None, None, None, Z.ZERO_F32,
                                              0, 64, Z.ZERO_F16, eps, 0.0, None, 0, None)


FLT_MAX = float.fromhex("0x1.fffffep127")


@pytest.mark.parametrize("call", [_norm_fwd, _joined_fwd])
def test_eps_is_finite_and_positive_in_binary32(Z, call):
    # above FLT_MAX a binary64 value rounds to inf, from half a step on; below half of the smallest subnormal, to 0
    for eps in (1e39, 1e300, float.fromhex("0x1.ffffffp127"), 2.0 ** 128, 2.0 ** -150, 5e-324):
        assert call(Z, eps) == Z._lib.ZERO_EINVAL, eps
    for eps in (FLT_MAX, float.fromhex("0x1.fffffefffffffp127"), 1e38, 2.0 ** -149, 1e-5):
        assert call(Z, eps) == Z._lib.ZERO_OK, eps


# ---- ResidualNorm -------------------------------------------------------------------------

def _place(Z, max_rows=16, cols=64):
    """A place with its buffers on the host: every call's checks run, none gets
    past the binding's check of the device."""
    import torch
    return Z.ResidualNorm(max_rows, cols, torch.ones(cols), dtype=torch.float32, device="cpu")


def test_a_refused_forward_leaves_the_last_one(Z):
    import torch
    place = _place(Z)
    place.rows = 3                                  # as a forward pass of 3 rows leaves it
    with pytest.raises(ValueError, match="device tensor"):
        place.forward(torch.zeros(5, 64))
    assert place.rows == 3 and place.r.shape == (3, 64)


@pytest.mark.parametrize("shape", [(2, 3, 32), (2, 1, 128), (64,) * 2 + (1,), (128,), ()])
def test_other_widths_are_not_taken_for_rows(Z, shape):
    """A batch whose last dimension is not the place's width is refused, also
    where its elements would fill whole rows."""
    import torch
    place = _place(Z, max_rows=4096)
    with pytest.raises(ValueError, match="64 columns"):
        place.forward(torch.zeros(shape))
    with pytest.raises(ValueError, match="64 columns"):
        place.forward(torch.zeros(6, 64), torch.zeros(shape))


def test_batches_of_other_lengths_are_not_taken_for_rows(Z):
    import torch
    place = _place(Z)
    for residual in (torch.zeros(2, 2, 64), torch.zeros(1, 7, 64)):
        with pytest.raises(ValueError):
            place.forward(torch.zeros(6, 64), residual)
    padded = torch.zeros(2, 3, 80)[:, :, :64]       # a batch of sequences inside wider rows: one matrix
    with pytest.raises(ValueError, match="device tensor"):
        place.forward(padded, padded)
