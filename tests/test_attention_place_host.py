"""A place is refused where it is made, not at its first pass."""
import pytest
import torch

from test_attention_host import Z  # noqa: F401  (fixture)


def test_types_that_attention_does_not_take(Z):  # noqa: F811
    for dtype in (torch.float32, torch.float64):
        with pytest.raises(ValueError, match="float16 or torch.bfloat16"):
            Z.WindowAttention(16, 4, 2, 8, dtype=dtype)
