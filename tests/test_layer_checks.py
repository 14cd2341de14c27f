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


# ---- the generator's state -------------------------------------------------------------------

class _State:
    """A generator state's face, on a device that need not be there."""
    is_cuda = True

    def __init__(self, device, nbytes=16):
        self._d, self._n, self.device = device, nbytes, f"cuda:{device}"

    def get_device(self):
        return self._d

    def numel(self):
        return self._n

    def element_size(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


class _Stream:
    cuda_stream = 0

    def __init__(self, device):
        self.device_index = device


@pytest.mark.parametrize("name", ["init", "advance"])
def test_generator_calls_refuse_other_devices(Z, monkeypatch, name):
    """The kernel would be enqueued on the current device's stream and write
    another device's memory."""
    import torch
    calls = []

    class Lib:
        def zero_rng_init(self, *a):
            calls.append(a)
            return 0

        def zero_rng_advance(self, *a):
            calls.append(a)
            return 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(Z._lib, "lib", lambda: Lib())
    monkeypatch.setattr(Z._lib, "_stream", lambda s: 0)
    call = (lambda t, s=None: Z.zero_rng_init(t, 1, stream=s)) if name == "init" else \
        (lambda t, s=None: Z.zero_rng_advance(t, stream=s))
    for bad in (lambda: call(_State(1)), lambda: call(_State(0), _Stream(1)), lambda: call(_State(0, 8)),
                lambda: call(torch.zeros(16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            bad()
    assert not calls
    call(_State(0))
    call(_State(0), _Stream(0))
    assert len(calls) == 2


def test_the_package_exports_every_entry_point(Z):
    """`from zero_partitioned_mixed_flatten_amd import *` has each function and constant of the binding."""
    public = {n for n in dir(Z) if n.startswith(("zero_", "ZERO_"))}
    assert public <= set(Z.__all__), public - set(Z.__all__)
    assert set(Z.__all__) <= set(dir(Z))
