"""Bias tables whose values lie far apart, in sequences that end inside a tile:
the rows past a sequence's end have distances that none of its pairs has, and
what the table holds for those must not come into the gradient of the bias."""
import pytest
import torch

from test_gpu_attention import BF16, F16, F32, Call

pytestmark = pytest.mark.gpu


def log(*a):
    print("[bias range]", *a, flush=True)


class Table(Call):
    """A call with one row of bias values for all heads."""

    def __init__(self, lengths, heads, kv_heads, dim, dtype, starts, values, bias_dtype, **kw):
        super().__init__(lengths, heads, kv_heads, dim, dtype, starts=starts, bias_dtype=bias_dtype, **kw)
        self.bias = torch.tensor([values] * heads, dtype=bias_dtype)
        self.dbias = self.bias.cuda()


# exp of the rise leaves binary32; the borders are past every distance of one sequence at least, and within 127 of them
CASES = [([1], [0, 1], [0.0, 100.0]),
         ([1, 5, 0, 3], [0, 1, 6], [-200.0, -100.0, 0.0]),
         ([1, 6, 70, 129], [0, 6], [-1000.0, 0.0]),
         ([280], [0, 285], [0.0, 150.0]),              # a wave past the end, wholly in the last bucket
         ([560], [0, 100, 600], [0.0, 1.0, 150.0]),    # the table, or at 64 columns a line a tile
         ([1050, 3], [0, 2, 1100], [0.0, 1.0, 150.0])]  # a line a tile


@pytest.mark.parametrize("case", range(len(CASES)))
def test_rows_past_the_end(case):
    lengths, starts, values = CASES[case]
    for dtype, dim, bias_dtype in ((F16, 64, F16), (BF16, 64, F32), (F16, 128, F32), (BF16, 128, BF16)):
        log(case, dtype, dim)
        c = Table(lengths, 2, 1, dim, dtype, starts, values, bias_dtype)
        got = c.check_bwd(*c.check_fwd())
        assert bool(got[3].isfinite().all())


def test_rows_past_the_end_off_16_byte_places():
    for window in (0, 3):
        c = Table([1, 6, 70], 2, 2, 64, F16, [0, 1, 6], [-300.0, -150.0, 0.0], F32, layout="odd", window=window)
        c.check_bwd(*c.check_fwd())
