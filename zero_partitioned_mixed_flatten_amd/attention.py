"""WindowAttention: the attention operators of one place in a transformer
block, wired to torch-owned device buffers.  Allocation and call order only;
the arithmetic is in the HIP kernels behind the C ABI.

The gradients a place produces (of the norms' weights and of the bias table)
are per-layer tensors that ShardStep.set_segments and AccumStep.plan take as
sources, or go straight to their place in the flat partition.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

from . import _lib as Z


class WindowAttention:
    """o = attention of the normed, turned queries and keys, for up to
    max_tokens tokens of packed sequences.

    wq, wk: weights of the norms over a head's dim elements (None: 1).  table:
    the rotation's angles (zero_rope_table), None: no rotation.  bias: heads x
    buckets, with starts the first distance of each bucket
    (zero_attention_buckets gives the usual ones); None: no bias.  Parameters
    are of the activations' type or float32; views into a shard's p16 or p32
    are fine at any offset.  window, sinks, scale: as attention_params.

    The forward pass keeps the queries and keys that it normed, the output and
    the rows' statistics for the backward pass, and uses the tensors it was
    given again there, so they stay as they are until then.  Those buffers and
    the workspace are fixed for the object's life: its calls are ordered on one
    stream."""

    def __init__(self, max_tokens: int, heads: int, kv_heads: int, dim: int, wq=None, wk=None, table=None, bias=None,
                 starts: Optional[Sequence[int]] = None, window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                 eps: float = 1e-6, interleaved: bool = False, max_sequences: int = 1, dtype=None, device="cuda"):
        import torch
        if max_tokens < 0 or max_sequences < 1:
            raise ValueError(f"WindowAttention: {max_tokens} tokens, {max_sequences} sequences")
        if (bias is None) != (starts is None):
            raise ValueError("WindowAttention: bias and starts go together")
        self.params = Z.attention_params(heads, kv_heads, dim, window, sinks, scale, starts)
        self.max_tokens, self.max_sequences = int(max_tokens), int(max_sequences)
        self.wq, self.wk, self.table, self.bias = wq, wk, table, bias
        self.eps, self.interleaved = float(eps), bool(interleaved)
        self.dtype = torch.float16 if dtype is None else dtype
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"WindowAttention: attention takes torch.float16 or torch.bfloat16, not {self.dtype}")
        new = lambda h: torch.empty(self.max_tokens, h, dim, dtype=self.dtype, device=self.device)
        self._q, self._k, self._o = new(heads), new(kv_heads), new(heads)
        self._lse = torch.empty(heads * self.max_tokens, dtype=torch.float32, device=self.device)
        # enough for fewer tokens or sequences, too
        need = max(16, Z.zero_qk_workspace_bytes(self.max_tokens, heads, kv_heads, dim),
                   Z.zero_attention_workspace_bytes(self.params, self.max_tokens, self.max_sequences))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        grad = lambda t: None if t is None else torch.zeros(t.shape, dtype=self.dtype, device=self.device)
        self.dwq, self.dwk, self.dbias = grad(wq), grad(wk), grad(bias)
        self._last = None

    @property
    def grads(self) -> Tuple:
        """The gradient tensors of (wq, wk, bias), in that order, without the absent ones."""
        return tuple(g for g in (self.dwq, self.dwk, self.dbias) if g is not None)

    def forward(self, q, k, v, o=None, offsets=None, sequences: int = 1, positions=None):
        """The attention's output for q (tokens, heads, dim) and k, v (tokens, kv_heads, dim): slices of a joint
        projection are fine.  offsets: int32 on the device, the sequences' first tokens and the end; None:
        `sequences` of equal length.  positions: of the tokens in their sequences (int32 on the device), needed with
        offsets and a rotation.  Rows outside all sequences go through the norms like others, so they need finite values
        and a position with angles; their rows of the place's own output are 0, those of a given o stay as they are."""
        tokens = q.shape[0]
        n = sequences if offsets is None else offsets.numel() - 1
        if tokens > self.max_tokens or n > self.max_sequences:
            raise ValueError(f"WindowAttention.forward: {tokens} tokens of {n} sequences, made for {self.max_tokens} of "
                             f"{self.max_sequences}")
        if self.table is not None and offsets is not None and positions is None:
            raise ValueError("WindowAttention.forward: packed sequences with a rotation need their positions")
        if offsets is None and (n < 1 or tokens % n):
            raise ValueError(f"WindowAttention.forward: {tokens} tokens are not {n} sequences of equal length")
        if self.table is not None and positions is None and tokens // n > self.table.shape[0]:
            raise ValueError(f"WindowAttention.forward: sequences of {tokens // n} tokens, angles of {self.table.shape[0]}")
        nq, nk = self._q[:tokens], self._k[:tokens]
        own = o is None
        o = self._o[:tokens] if own else o
        lse = self._lse[:self.params.heads * tokens].view(self.params.heads, tokens)
        turn = dict(eps=self.eps, positions=positions, period=0 if offsets is not None else tokens // n,
                    interleaved=self.interleaved)
        where = dict(offsets=offsets, sequences=n)
        self._last = None                           # the buffers are the new call's from here on
        if own and offsets is not None:
            Z.zero_attention_clear_rows(o, offsets)
        Z.zero_qk_norm_rope_fwd(nq, nk, q, k, self.wq, self.wk, self.table, **turn)
        Z.zero_attention_fwd(o, lse, nq, nk, v, self.params, bias=self.bias, **where)
        self._last = (q, k, v, nq, nk, o, lse, turn, where)
        return o

    def backward(self, dout, dq=None, dk=None, dv=None, grads=None, accumulate: bool = False):
        """(dq, dk, dv): the gradients at the last forward pass's q, k and v from the output's.  The parameters' go to
        self.dwq, self.dwk and self.dbias, or to `grads`, three tensors (None: not wanted) such as slices of a
        partition; accumulate adds them to what is there.  In rows outside all sequences dq and dk are 0, and so is dv
        where it is made here; those of a given dv stay as they are."""
        import torch
        if self._last is None:
            raise ValueError("WindowAttention.backward: no forward pass")
        q, k, v, nq, nk, o, lse, turn, where = self._last
        new = lambda t: torch.empty(t.shape, dtype=self.dtype, device=self.device)
        own_dv = dv is None
        dq, dk, dv = new(q) if dq is None else dq, new(k) if dk is None else dk, new(v) if own_dv else dv
        for t in (dq, dk, dv):
            if t.numel() and any(t.data_ptr() == x.data_ptr() for x in (q, k, v, o, dout)):
                raise ValueError("WindowAttention.backward: a gradient over a tensor that is still read")
        if where["offsets"] is not None:            # rows outside all sequences: nothing for the norms' gradients
            for t in (dq, dk, dv) if own_dv else (dq, dk):
                Z.zero_attention_clear_rows(t, where["offsets"])
        dwq, dwk, dbias = (self.dwq, self.dwk, self.dbias) if grads is None else grads
        Z.zero_attention_bwd(dq, dk, dv, dbias, dout, o, lse, nq, nk, v, self.params, bias=self.bias, accumulate=accumulate,
                             workspace=self.workspace, **where)
        Z.zero_qk_norm_rope_bwd(dq, dk, dwq, dwk, dq, dk, q, k, self.wq, self.wk, self.table, accumulate=accumulate,
                                workspace=self.workspace, **turn)
        return dq, dk, dv
