"""Sizes past what one dimension of a launch holds: 2^24 workgroups of 256."""
import pytest
import torch

import attention_oracle as A
from test_gpu_attention import F16, close

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402


def test_more_heads_than_one_dimension_of_a_launch():
    """4200 tokens of 65535 heads of 256, 16 heads a workgroup: 2^24.04.  Head h of token i is row i + h of a small matrix, in the
    output, too: without a rotation they are the same values."""
    tokens, heads, dim = 4200, 65535, 256
    g = torch.Generator().manual_seed(8)
    x = torch.randn(tokens + heads, dim, generator=g).half()
    w = (1.0 + 0.1 * torch.randn(dim, generator=g)).half()
    dev = x.cuda()
    out = torch.zeros_like(dev)
    view = lambda t: torch.as_strided(t, (tokens, heads, dim), (dim, dim, 1))
    Z.zero_qk_norm_rope_fwd(view(out), None, view(dev), None, w.cuda(), None, None)
    want, e = A.qk_fwd(x[:-1, None].double(), w.double(), None, 1e-6, False)
    close(out[:-1, None], want, A.stored(e, want, F16), "y")
    assert bool((out[-1] == 0).all())


def test_a_table_past_one_dimension_of_a_launch():
    """2^25 + 5 positions of 128 pairs: 2^32 entries and more."""
    n = (1 << 25) + 5
    table = torch.zeros(n, 128, 2, device="cuda")
    Z.zero_rope_table(table)
    at = torch.tensor([0, 1, 1000003, 1 << 24, (1 << 25) - 1, 1 << 25, n - 1])
    want = A.angles(at, 256, 10000.0)
    # half a step of 1, and a binary64 angle of up to 2^25 at 2^-53 relatively, a few times
    close(table[at.cuda()], want, 2.0 ** -24 + 16 * 2.0 ** -28 + 0 * want, "table")
