"""The layer operators together with the shard step that consumes their
gradients: a residual stream of several places whose parameters are views of
the shard's fp16 copy, their gradients flattened (or added straight into the
fp32 partition), the exact norm, the decision and the update -- against the
64-bit forms layer by layer and the oracle's step bit for bit."""
import numpy as np
import pytest
import torch

import layer_oracle as L
import oracle as O

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402

SEED = 0xFEEDFACECAFE


def log(*a):
    print("[layer step]", *a, flush=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, want, bound, what):
    bad = ~(np.abs(f64(got) - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.abs(f64(got) - want).max())


def check_place(place, x, res, y, dy, dres, dx, dr, step, kind="f16"):
    """One place's forward and backward pass against the 64-bit forms, from the
    device's own inputs and stored r."""
    rows, cols = x.shape
    kept, s = L.keep(rows, cols, place.p, SEED, step, place.site), L.scale(place.p)
    v = x.cpu().float() + place.bias.cpu().float()
    v = res.cpu().float() + torch.where(torch.from_numpy(kept), v * np.float32(s), torch.zeros(()))
    assert torch.equal(place.r.cpu(), v.half())
    want, bound = L.norm_fwd(f64(place.r), f64(place.w)[None], f64(place.b)[None], place.eps, kind)
    close(y, want[0], bound[0], "y")
    mean, rstd = f64(place._mean[:rows]), f64(place._rstd[:rows])
    want, bound = L.norm_bwd(f64(dy), f64(place.r), mean, rstd, f64(place.w)[None], f64(dres))
    e, e_e = want[0], 1.01 * bound[0]
    close(dr, e, L.stored(e_e, e, kind), "dr")
    d = L.dropped(e, kept, s)
    e_d = L.dropped(e_e, kept, s) + L.U * np.abs(d)
    close(dx, d, L.stored(e_d, d, kind), "dx")
    total, e_t = L.column_sum(d, e_d)
    return [(want[1], bound[1]), (want[2], bound[2]), (total, e_t)]


class Stream:
    """`depth` places in a row over a shard holding their parameters (each
    place's bias, norm weight and norm bias, the odd width leaving them at odd
    offsets) and nothing else."""

    def __init__(self, depth, rows, cols, step):
        self.cols, self.rng = cols, Z.LayerRng(SEED)
        self.step = step
        n = 3 * depth * cols
        g = np.random.default_rng(5)
        p = np.empty((depth, 3, cols), np.float32)
        p[:, 0] = 0.1 * g.standard_normal((depth, cols))
        p[:, 1] = 1.0 + 0.1 * g.standard_normal((depth, cols))
        p[:, 2] = 0.1 * g.standard_normal((depth, cols))
        self.p32 = p.reshape(-1)
        step.p32.copy_(torch.from_numpy(self.p32))
        step.p16.copy_(step.p32.half())
        view = lambda i: step.p16[i * cols:(i + 1) * cols]
        self.places = [Z.ResidualNorm(rows, cols, view(3 * k + 1), view(3 * k + 2), view(3 * k), p=0.1, rng=self.rng, site=k)
                       for k in range(depth)]
        assert n == step.n

    def forward(self, h, r):
        """h: the sublayer's output, r: the residual stream."""
        self.inputs, self.outputs = [], []
        for place in self.places:
            self.inputs.append((h, r))
            h = place.forward(h, r)
            self.outputs.append(h)
            r = place.r
            h = (h * 0.5).half()                    # stands for the sublayer between two places
        return h, r

    def backward(self, dy, dres, **kw):
        self.grads_in, self.grads_out = [None] * len(self.places), [None] * len(self.places)
        for k in reversed(range(len(self.places))):
            self.grads_in[k] = (dy, dres)
            k_kw = {a: v[k] if a == "grads" else v for a, v in kw.items()}
            dx, dr = self.places[k].backward(dy, dres, **k_kw)
            self.grads_out[k] = (dx, dr)
            dy, dres = (dx * 0.5).half(), dr
        return dy, dres


def test_training_steps_through_the_flatten():
    """Three steps: forward, backward, flatten of the places' gradient tensors,
    exact norm, decision, update, generator advanced.  The second step's
    gradients overflow binary16: it is skipped, the scale halves and the
    parameters stay."""
    depth, rows, cols = 3, 257, 203
    n = 3 * depth * cols
    step = Z.ShardStep(n, fused=True)
    net = Stream(depth, rows, cols, step)
    segs, srcs = [], []
    for k, place in enumerate(net.places):
        for j, t in enumerate((place.dbias, place.dw, place.db)):
            segs.append((len(srcs), 0, (3 * k + j) * cols, cols))
            srcs.append(t)
    step.set_segments(srcs, segs)
    scale0 = 1024.0
    step.init_state(scale0)
    st_o, hp_o, hp = O.new_state(scale0), O.hparams(), Z.hparams()
    p32, m, v = net.p32.copy(), np.zeros(n, np.float32), np.zeros(n, np.float32)
    p16 = p32.astype(np.float16).view(np.uint16)
    g = torch.Generator()
    g.manual_seed(11)
    for k in range(3):
        log("step", k)
        scale = step.read_state().loss_scale
        assert scale == st_o.loss_scale == (scale0 if k < 2 else scale0 / 2)
        h0, r0 = (torch.randn(rows, cols, generator=g).half().cuda() for _ in range(2))
        big = 500.0 if k == 1 else 1e-3             # times the scale: the second step's sums pass 65504
        dy = (torch.randn(rows, cols, generator=g) * big * scale / 16).clamp(-3e4, 3e4).half().cuda()
        dres = (torch.randn(rows, cols, generator=g) * 1e-3 * scale).half().cuda()
        net.forward(h0, r0)
        net.backward(dy, dres)
        torch.cuda.synchronize()
        for i, place in enumerate(net.places):
            if k == 1:
                break
            (x, res), (gy, gres), (dx, dr) = net.inputs[i], net.grads_in[i], net.grads_out[i]
            want = check_place(place, x, res, net.outputs[i], gy, gres, dx, dr, step=k)
            for got, (t, e) in zip((place.dw, place.db, place.dbias), want):
                close(got, t, L.stored(e, t, "f16"), "parameter gradient")
        step.step(hp)
        net.rng.advance()
        torch.cuda.synchronize()
        grads = [s.cpu().numpy().view(np.uint16) for s in srcs]
        grad_o = np.empty(n, np.uint16)
        O.step(hp_o, st_o, grads, segs, grad_o, p16, p32, m, v)
        s = step.read_state()
        assert (s.skip, s.loss_scale, s.step, s.sumsq) == (st_o.skip, st_o.loss_scale, st_o.step, st_o.sumsq)
        assert s.skip == (1 if k == 1 else 0)
        assert np.array_equal(step.grad16.cpu().numpy().view(np.uint16), grad_o)
        assert np.array_equal(step.p16.cpu().numpy().view(np.uint16), p16)
        assert np.array_equal(step.p32.cpu().numpy(), p32) and np.array_equal(step.v32.cpu().numpy(), v)
        assert step.guard_intact()
    assert net.rng.read().step == 3


def test_accumulation_straight_into_the_partition():
    """Two micro-batches: the places add their gradients straight to their
    slices of the fp32 partition (the first one stores), which then holds
    their sum; the norm, the decision and the update read it as ever."""
    depth, rows, cols = 2, 130, 77
    n = 3 * depth * cols
    step = Z.AccumStep(n, fused=False)
    net = Stream(depth, rows, cols, step)
    step.init_state(256.0)
    step.grad32.fill_(float("nan"))                 # the first micro-batch stores, it does not add
    cut = lambda i: step.grad32[i * cols:(i + 1) * cols]
    slices = [(cut(3 * k + 1), cut(3 * k + 2), cut(3 * k)) for k in range(depth)]
    g = torch.Generator()
    g.manual_seed(3)
    total, bound = np.zeros(n), np.zeros(n)
    for mb in range(2):
        log("micro-batch", mb)
        rows_mb = rows - 41 * mb                    # the second one is shorter
        h0, r0, dy, dres = (torch.randn(rows_mb, cols, generator=g).half().cuda() for _ in range(4))
        net.forward(h0, r0)
        net.backward(dy, dres, grads=slices, accumulate=mb > 0)
        torch.cuda.synchronize()
        for i, place in enumerate(net.places):
            (x, res), (gy, gres), (dx, dr) = net.inputs[i], net.grads_in[i], net.grads_out[i]
            want = check_place(place, x, res, net.outputs[i], gy, gres, dx, dr, step=mb)
            for j, (t, e) in zip((1, 2, 0), want):
                at = slice((3 * i + j) * cols, (3 * i + j + 1) * cols)
                total[at] += t
                bound[at] += 1.01 * e + L.U * np.abs(total[at])
        net.rng.advance()
    close(step.grad32[:n], total, bound, "accumulated gradients")
    grad = step.grad32.cpu().numpy().copy()
    st_o, hp_o, hp = O.new_state(256.0), O.hparams(), Z.hparams()
    p32, m, v = net.p32.copy(), np.zeros(n, np.float32), np.zeros(n, np.float32)
    p16 = p32.astype(np.float16).view(np.uint16)
    step.norm_overflow(hp)
    step.adam()
    torch.cuda.synchronize()
    O.decide(st_o, hp_o, *O.norm_overflow_f32(grad))
    O.adam_update_f32(st_o, p16, p32, m, v, grad)
    assert step.read_state().sumsq == st_o.sumsq
    assert np.array_equal(step.p16.cpu().numpy().view(np.uint16), p16)
    assert np.array_equal(step.p32.cpu().numpy(), p32)
    assert step.guard_intact()


def test_recomputed_forward_is_the_same():
    """Activation checkpointing: the forward pass run again for the backward
    pass gives the same r, y and statistics bit for bit, from the generator's
    counters alone."""
    rows, cols = 300, 1600
    w, b, bias = (torch.randn(cols, device="cuda").half() for _ in range(3))
    rng = Z.LayerRng(SEED)
    place = Z.ResidualNorm(rows, cols, w, b, bias, p=0.3, rng=rng, site=4)
    x, res = (torch.randn(2, 150, cols, device="cuda").half() for _ in range(2))
    y = place.forward(x, res)
    r, mean = place.r.clone(), place._mean.clone()
    y2 = place.forward(x, res)
    log("recompute")
    assert torch.equal(y, y2) and torch.equal(r, place.r) and torch.equal(mean, place._mean)
    rng.advance()
    place.forward(x, res)
    assert not torch.equal(r, place.r)


def test_fewer_rows_and_refusals():
    w = torch.ones(64, device="cuda").half()
    place = Z.ResidualNorm(16, 64, w)
    x = torch.randn(5, 64, device="cuda").half()
    y = place.forward(x)                            # no residual, bias, or dropout: the layer norm of x
    assert y.shape == (5, 64) and torch.equal(place.r, x) and len(place.grads) == 1
    dx, dr = place.backward(torch.ones_like(y))
    assert torch.equal(dx, dr)                      # nothing dropped
    with pytest.raises(ValueError, match="made for 16"):
        place.forward(torch.zeros(17, 64, device="cuda").half())
    with pytest.raises(Z.ZeroError):                # dropout without a generator
        Z.ResidualNorm(16, 64, w, p=0.1).forward(x)
    with pytest.raises(TypeError):
        place.forward(x.float())
