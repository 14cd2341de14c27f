"""ResidualNorm: the layer operators of one place in a transformer block's
residual stream, wired to torch-owned device buffers, and LayerRng, the state
of the dropout generator.  Allocation and call order only; the arithmetic is
in the HIP kernels behind the C ABI.

The gradients a place produces (of its norm's weight and bias and of the bias
before it: ln1, ln2, ln_f and the projections' biases of a GPT block) are
per-layer tensors that ShardStep.set_segments and AccumStep.plan take as
sources, or go straight to their place in the flat partition.
"""
from __future__ import annotations

from typing import Optional, Tuple

from . import _lib as Z


class LayerRng:
    """A dropout generator: 16 bytes of device memory holding the seed and a
    count of passes.  One generator serves every ResidualNorm of a model (each
    has its own site); advance() after each backward pass, inside the captured
    graph where there is one.  A training step of several micro-batches
    (AccumStep) advances after each of them: masks are a function of the seed,
    the count, the site and the element, so micro-batches under one count would
    all drop the same elements.  Ranks that train on different data take
    different seeds for the same reason."""

    def __init__(self, seed: int, device="cuda"):
        import torch
        self.state = torch.zeros(Z.RNG_BYTES, dtype=torch.uint8, device=device)
        Z.zero_rng_init(self.state, seed)

    def advance(self) -> None:
        Z.zero_rng_advance(self.state)

    def read(self) -> Z.RngState:
        return Z.read_rng(self.state)


class ResidualNorm:
    """r = residual + D(x + bias); y = layer norm of r, for up to max_rows rows
    (tokens) of cols columns.

    w, b, bias: parameter vectors on the device, of the activations' type or
    float32; views into a shard's p16 or p32 are fine at any offset (the step
    then updates the layer in place).  b and bias may be None.  The forward
    pass keeps r and the rows' statistics for the backward pass; those buffers
    and the workspace are fixed for the object's life, so its calls are ordered
    on one stream."""

    def __init__(self, max_rows: int, cols: int, w, b=None, bias=None, p: float = 0.0, rng: Optional[LayerRng] = None,
                 site: int = 0, eps: float = 1e-5, dtype=None, device="cuda"):
        import torch
        if max_rows < 0 or cols < 1:
            raise ValueError(f"ResidualNorm: {max_rows} rows of {cols} columns")
        self.cols, self.w, self.b, self.bias = int(cols), w, b, bias
        self.p, self.rng, self.site, self.eps = float(p), rng, int(site), float(eps)
        self.dtype = torch.float16 if dtype is None else dtype
        self.device = torch.device(device)
        self.max_rows = int(max_rows)
        self._r = torch.empty(self.max_rows, self.cols, dtype=self.dtype, device=self.device)
        self._mean = torch.empty(self.max_rows, dtype=torch.float32, device=self.device)
        self._rstd = torch.empty(self.max_rows, dtype=torch.float32, device=self.device)
        # no fewer rows ever need more than max_rows do
        self.workspace = torch.empty(max(16, Z.zero_layer_workspace_bytes(self.max_rows, self.cols)),
                                     dtype=torch.uint8, device=self.device)
        grad = lambda t: None if t is None else torch.zeros(self.cols, dtype=self.dtype, device=self.device)
        self.dw, self.db, self.dbias = grad(w), grad(b), grad(bias)
        self.rows = 0

    @property
    def r(self):
        """The residual stream the last forward pass stored (its rows)."""
        return self._r[:self.rows]

    @property
    def grads(self) -> Tuple:
        """The gradient tensors of (w, b, bias), in that order, without the absent ones."""
        return tuple(g for g in (self.dw, self.db, self.dbias) if g is not None)

    def _matrix(self, t, rows):
        """A batch of any number of dimensions, the last of them the columns, as a matrix."""
        if t.dim() < 1 or t.shape[-1] != self.cols or t.numel() != rows * self.cols:
            raise ValueError(f"ResidualNorm.forward: expected {rows} rows of {self.cols} columns, got {tuple(t.shape)}")
        return t if t.dim() == 2 else t.view(rows, self.cols)

    def forward(self, x, residual=None, y=None):
        """y of the rows of x (any shape whose last dimension is the columns); r
        stays in self.r."""
        import torch
        rows = x.numel() // self.cols
        if rows > self.max_rows:
            raise ValueError(f"ResidualNorm.forward: {rows} rows, made for {self.max_rows}")
        x = self._matrix(x, rows)
        residual = None if residual is None else self._matrix(residual, rows)
        if y is None:
            y = torch.empty(rows, self.cols, dtype=self.dtype, device=self.device)
        Z.zero_dropout_layernorm_fwd(self._r[:rows], y, self._mean[:rows], self._rstd[:rows], x, residual, self.bias,
                                     self.w, self.b, self.eps, self.p, self.rng.state if self.rng else None, self.site)
        self.rows = rows                            # a refused call leaves the last one's
        return y

    def backward(self, dy, dres=None, dx=None, dr=None, grads=None, accumulate: bool = False):
        """(dx, dr): the gradients at x and at the residual, from y's and (dres)
        r's own.  The parameters' go to self.dw, self.db and self.dbias, or to
        `grads`, three vectors (None: not wanted) such as slices of a
        partition; accumulate adds them to what is there."""
        import torch
        rows = self.rows
        new = lambda: torch.empty(rows, self.cols, dtype=self.dtype, device=self.device)
        dx, dr = new() if dx is None else dx, new() if dr is None else dr
        dw, db, dbias = (self.dw, self.db, self.dbias) if grads is None else grads
        Z.zero_dropout_layernorm_bwd(dx, dr, dw, db, dbias, dy, dres, self.r, self._mean[:rows], self._rstd[:rows],
                                     self.w, self.p, self.rng.state if self.rng else None, self.site, accumulate,
                                     self.workspace)
        return dx, dr
