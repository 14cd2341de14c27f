"""Buckets that a bias masks: -inf, the type's lowest value, -1e9.  Their pairs
have no weight and no gradient, and those of the other buckets are what they are
without them."""
import math

import pytest
import torch

from test_gpu_attention import BF16, F16, F32, Call

pytestmark = pytest.mark.gpu


class Masked(Call):
    """`masked` buckets hold `value` on the device and, for the 64-bit form, -1e30, whose weights are 0 as well."""

    def __init__(self, lengths, dim, dtype, starts, masked, value, bias_dtype, **kw):
        super().__init__(lengths, 4, 2, dim, dtype, starts=starts, bias_dtype=bias_dtype, **kw)
        self.bias[:, masked] = value
        self.dbias = self.bias.cuda()
        self.bias = self.bias.double()
        self.bias[:, masked] = -1e30

    def bwd(self, o, lse, grad_dtype=None, accumulate=False, start=0.0, workspace=None):
        return super().bwd(o, lse, self.dbias.dtype, accumulate, start, workspace)


@pytest.mark.parametrize("value", ["inf", "lowest", "1e9"])
@pytest.mark.parametrize("starts,lengths", [([0, 2, 5, 9, 40], [300, 1, 70]), ([0, 2, 5, 9, 1100], [1300, 40]), ([0, 2, 5, 9, 600], [700, 40])])
def test_masked_buckets(starts, lengths, value):
    for dtype, dim, bias_dtype in ((F16, 64, F16), (BF16, 64, BF16), (F16, 128, F32), (BF16, 128, F32)):
        if value == "1e9" and bias_dtype is F16:
            continue
        print("[masked buckets]", starts, value, dtype, dim, flush=True)
        v = {"inf": -math.inf, "lowest": torch.finfo(bias_dtype).min, "1e9": -1e9}[value]
        for masked in ([1, 4], [2], [1, 2, 3, 4]):
            c = Masked(lengths, dim, dtype, starts, masked, v, bias_dtype)
            got = c.check_bwd(*c.check_fwd())
            assert bool((got[3][:, masked] == 0).all())
