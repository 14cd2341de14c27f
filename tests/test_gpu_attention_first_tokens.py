"""Gradients at first tokens that stay visible, in batches where some sequences
have queries behind the window and others do not: the former's are summed apart,
in the workspace and nowhere beside it."""
import pytest
import torch

from test_gpu_attention import BF16, F16, Call

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402

W = 70                                                    # from 70 + 128 tokens on a sequence has queries behind the window


class Bounded(Call):
    """With a workspace of just the size, and sentinels behind it."""

    def bwd(self, o, lse, *args, **kw):
        n = self.where["sequences"] if "sequences" in self.where else self.where["offsets"].numel() - 1
        need = Z.zero_attention_workspace_bytes(self.params, self.tokens, n)
        ws = torch.full((need + 4096,), 0x7E, dtype=torch.uint8, device="cuda")
        out = super().bwd(o, lse, *args, workspace=ws[:need], **kw)
        assert bool((ws[need:] == 0x7E).all())
        return out


CASES = [[197, 198, 199], [1, 197, 0, 1, 1200, 5, 197], [198] * 7, [1, 198, 1, 198, 1], [40] * 12 + [2000] + [40] * 3, [10, 1024 + 197, 3, 1024 + 198, 9],
         [128] * 5, [3000, 1]]


@pytest.mark.parametrize("lengths", CASES, ids=lambda c: "-".join(map(str, c[:4])))
@pytest.mark.parametrize("heads,kv_heads", [(2, 1), (3, 3)])
def test_long_and_short_sequences(lengths, heads, kv_heads):
    for dtype, dim in ((F16, 64), (BF16, 128)):
        print("[first tokens]", lengths, heads, dim, flush=True)
        c = Bounded(lengths, heads, kv_heads, dim, dtype, window=W, sinks=3, after=2)
        c.check_bwd(*c.check_fwd())


@pytest.mark.parametrize("n,seqs", [(197, 4), (198, 4), (199, 3), (1221, 2), (1223, 2)])
def test_equal_lengths(n, seqs):
    for dtype, dim in ((F16, 64), (BF16, 128)):
        print("[first tokens]", n, seqs, dim, flush=True)
        c = Bounded([n] * seqs, 2, 1, dim, dtype, window=W, sinks=128, equal=True)
        c.check_bwd(*c.check_fwd())


def test_enough_sequences_for_one_part_a_piece():
    """So many pieces of keys that none is cut into parts: the long sequences' first ones alone go through the workspace."""
    lengths = [33, 250, 7, 198, 64, 197] * 12
    c = Bounded(lengths, 8, 8, 64, F16, window=W, sinks=5, after=3)
    c.check_bwd(*c.check_fwd())
    c = Bounded([230] * 40, 8, 8, 64, BF16, window=W, sinks=5, equal=True)
    c.check_bwd(*c.check_fwd())


def test_offsets_out_of_order():
    """Whatever the offsets hold, nothing outside the outputs and the workspace is written."""
    c = Bounded([500, 500], 2, 1, 64, F16, window=W, sinks=2, layout="odd", after=3)
    o, lse = c.fwd()
    for bad in ([0, 5, 2], [-7, 500, 10 ** 9], [1003, 0, 400], [900, 30, 1003], [2 ** 31 - 1, -2 ** 31, 0], [0, 1003, 0]):
        print("[first tokens] offsets", bad, flush=True)
        c.where = {"offsets": torch.tensor(bad, dtype=torch.int32, device="cuda")}
        c.end = c.tokens
        c.bwd(o, lse)
