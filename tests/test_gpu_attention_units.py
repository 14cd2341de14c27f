"""binary16's exponents in the attention kernels: keys with weights far below
the row's largest, which are many."""
import math

import pytest
import torch

import attention_oracle as A
from test_gpu_attention import BF16, F16, Call, close

pytestmark = pytest.mark.gpu


class Far(Call):
    """One head: the first key takes all but exp(-gap) a key of every later query's weight.  q = a e0, k_0 = 32 e0, the other
    keys 8 e2; v_0 = 0, the other values 64 e1; do = g e1."""

    def __init__(self, n, dim, dtype, gap, g=1.0):
        super().__init__([n], 1, 1, dim, dtype, scale=0.125)
        for t in (self.q, self.k, self.v, self.do):
            t.zero_()
        self.gap = gap
        self.q[:, 0, 0] = gap / 4.0
        self.k[0, 0, 0] = 32.0
        self.k[1:, 0, 2] = 8.0
        self.v[1:, 0, 1] = 64.0
        self.do[:, 0, 1] = g
        for name in ("q", "k", "v", "do"):
            self.d[name].copy_(getattr(self, name))


N = 40000


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_many_small_weights(dtype, dim):
    """40000 keys of weight 2^-26: together 6e-4 of a row, 0.04 of its output, and each less than half of binary16's smallest
    number beside the largest weight."""
    c = Far(N, dim, dtype, 18.0)
    o, lse = c.fwd()
    i = torch.arange(N, dtype=torch.float64)
    w = i * math.exp(-18.0)
    want = torch.zeros(N, dim, dtype=torch.float64)
    want[:, 1] = 64.0 * w / (1.0 + w)
    # a weight and its row's sum: half a step of the weight; binary32's roundings of the score (gap 18: 8 u 18), its exponential
    # (8 u) and a sum of n terms (2 n u), and of the product's sum the same; binary16 below 2^-14 off by 2^-25, of weights in
    # units of 2^-7.  lse: the sum is 1 + w, of a lane's 32 terms of a tile first, then of its tiles: 2 (32 + n / 64 + 2) u of it
    e = want * (A.HALF[dtype] + (8 * 18 + 16 + 2 * 2 * N) * A.U)
    if dtype == F16:
        e[:, 1] += i * 2.0 ** -32 * 64.0
    close(o[:, 0], want, A.stored(e, want, dtype), "o")
    close(lse[0], 18.0 + torch.log1p(w), 18.0 * 8 * A.U + 2 * (34 + N / 64) * A.U + 16 * A.U + 0 * w, "lse")
