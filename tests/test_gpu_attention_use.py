"""The attention operators as a program uses them: a place of a block through
WindowAttention with its gradients in a ShardStep, streams and captured graphs,
equal calls, inf and NaN in rows that others do not see, batches without
tokens, offsets past 2^32 elements."""
import math

import numpy as np
import pytest
import torch

import attention_oracle as A
import oracle as O
from test_gpu_attention import BF16, F16, F32, SENTINEL, STARTS, Call, close

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402

U = A.U


def log(*a):
    print("[attention use]", *a, flush=True)


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


def test_equal_calls_give_equal_bits():
    for starts, dim, kv in ((STARTS["logs"], 64, 5), (STARTS["wide"], 128, 1), (None, 128, 5)):
        c = Call([700, 30, 1300], 5, kv, dim, F16, window=300, sinks=5, starts=starts, bias_dtype=F32 if starts else None)
        o, lse = c.fwd()
        first = c.bwd(o, lse)
        noise = torch.randn(4096, 4096, device="cuda")
        for _ in range(3):
            noise @ noise
            assert same(c.fwd(), (o, lse)) and same(c.bwd(o, lse), first)


def test_workspace_contents_do_not_matter():
    c = Call([900, 200], 4, 2, 64, F16, window=200, sinks=3, starts=STARTS["logs"])
    o, lse = c.fwd()
    need = Z.zero_attention_workspace_bytes(c.params, c.tokens, 2)
    want = c.bwd(o, lse)
    for fill in (0xFF, 0x7C, 0):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert same(c.bwd(o, lse, workspace=ws), want)
    ws = torch.full((need + 64,), 0x55, dtype=torch.uint8, device="cuda")
    assert same(c.bwd(o, lse, workspace=ws[:need]), want) and bool((ws[need:] == 0x55).all())
    with pytest.raises(Z.ZeroError):
        c.bwd(o, lse, workspace=ws[:need - 1])


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_rows_do_not_see_later_ones(value):
    """inf and NaN from some token on: the rows before are what they are without them, within the bounds.  (Not bit for
    bit: the rows of a wave raise the base that their sums go by together, when one of them has to, and a sum's roundings
    go by its base; the bounds hold for any base.)"""
    for dtype, dim, starts in ((F16, 64, None), (BF16, 128, STARTS["logs"]), (F16, 80, STARTS["far"])):
        for lengths, bad in (([300], 150), ([200, 100], 260)):
            log("later", value, dtype, dim, lengths)
            c = Call(lengths, 3, 1, dim, dtype, starts=starts)
            o, lse = c.fwd()
            for name in ("q", "k", "v"):
                c.d[name][bad:] = value
            o2, lse2 = c.fwd()
            first = 128 if lengths[0] == 300 else 200              # up to here no wave has a row with such a value
            assert torch.equal(o2[:first], o[:first]) and torch.equal(lse2[:, :first], lse[:, :first])
            (want, wl), (e, el) = c.want_fwd()
            close(o2[:bad], want[:bad], A.stored(e, want, dtype)[:bad], "o")
            close(lse2[:, :bad], wl[:, :bad], (el + A.stored(0 * el, wl, F32))[:, :bad], "lse")
            assert bool(o2[bad:].isnan().any())


def test_rows_behind_the_window_are_not_seen():
    c = Call([400], 2, 2, 64, F16, window=50, sinks=2)
    (want, _), (e, _) = c.want_fwd()
    for name in ("k", "v"):
        c.d[name][10:100] = math.nan
    o, _ = c.fwd()
    keep = torch.ones(400, dtype=torch.bool)
    keep[10:149] = False                            # 149 sees 100 on
    close(o[keep.cuda()], want[keep], A.stored(e, want, F16)[keep], "o")
    assert bool(o[10:149].isnan().flatten(1).any(1).all())


def test_rows_long_behind_first_tokens_and_window():
    """The same with keys between the first tokens and the window's, whole tiles of them, and one such value that is seen."""
    for value in (math.nan, math.inf):
        c = Call([700], 2, 1, 128, BF16, window=50, sinks=70)
        (want, _), (e, _) = c.want_fwd()
        c.d["k"][400:460] = value
        c.d["v"][400:460] = value
        c.d["v"][600, 0, 5] = value
        o, _ = c.fwd()
        keep = torch.ones(700, dtype=torch.bool)
        keep[400:509] = False                        # 509 sees 460 on
        keep[600:650] = False
        close(o[keep.cuda()], want[keep], A.stored(e, want, BF16)[keep], "o")
        bad = o[600:650]
        assert bool(bad[:, :, 5].isfinite().logical_not().all()) and bool(bad[:, :, :5].isfinite().all())
        assert bool(bad[:, :, 6:].isfinite().all())


def test_other_sequences_do_not_matter():
    """Whatever one sequence and the rows behind the last hold, the others' results and gradients are the same bits."""
    c = Call([130, 70, 200], 4, 2, 64, F16, window=90, sinks=3, after=9)
    o, lse = c.fwd()
    g = c.bwd(o, lse)
    for value in (math.nan, math.inf, 60000.0):
        for name in ("q", "k", "v", "do"):
            c.d[name][130:200] = value
            c.d[name][400:] = value
        o2, lse2 = c.fwd()
        o2[130:200], lse2[:, 130:200] = o[130:200], lse[:, 130:200]
        keep = [slice(0, 130), slice(200, 400)]
        g2 = c.bwd(o2, lse2)
        for s in keep:
            assert torch.equal(o2[s], o[s]) and torch.equal(lse2[:, s], lse[:, s])
            assert all(torch.equal(a[s], b[s]) for a, b in zip(g2[:3], g[:3]))


def test_large_scores():
    """Scores far from 0 and far apart: the maximum is taken off before they are raised."""
    for spread in (6.0, 20.0):
        c = Call([333], 2, 1, 64, BF16, spread=spread)
        c.check_fwd()
        c = Call([333], 2, 1, 64, F16, spread=spread, scale=1.0 / 64)
        c.check_fwd()
    c = Call([256], 1, 1, 64, BF16)                 # scores that rise from tile to tile, and fall
    for sign in (1.0, -1.0):
        c.k[:] = 0.0
        c.k[:, 0, 0] = sign * torch.arange(256).bfloat16()
        c.q[:, 0, 0] = 8.0
        c.d["k"].copy_(c.k)
        c.d["q"].copy_(c.q)
        c.check_fwd()


def test_two_streams():
    calls = [Call([500, 77], 4, 2, 64, F16, window=100, sinks=1, starts=STARTS["logs"], seed=i) for i in range(2)]
    want = []
    for c in calls:
        o, lse = c.fwd()
        want.append((o, lse, c.bwd(o, lse)))
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = []
        for c, s in zip(calls, streams):
            s.wait_stream(torch.cuda.current_stream())
            o, lse = torch.empty_like(c.d["q"]), torch.empty(c.hq, c.tokens, device="cuda")
            outs = [torch.empty_like(c.d[n]) for n in ("q", "k", "v")] + [torch.empty_like(c.dbias)]
            torch.cuda.synchronize()
            Z.zero_attention_fwd(o, lse, c.d["q"], c.d["k"], c.d["v"], c.params, bias=c.dbias, stream=s, **c.where)
            Z.zero_attention_bwd(*outs, c.d["do"], o, lse, c.d["q"], c.d["k"], c.d["v"], c.params, bias=c.dbias, stream=s, **c.where)
            got.append((o, lse, outs))
        torch.cuda.synchronize()
        for (o, lse, g), (wo, wl, wg) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl) and same(g, wg)


def test_captured_graphs():
    """Two graphs of the whole place, each with its own buffers, replayed in turn over new inputs with eager work between."""
    torch.manual_seed(3)
    T, hq, hk, d = 333, 6, 2, 64
    table = torch.empty(T, d // 2, 2, device="cuda")
    Z.zero_rope_table(table)
    places, graphs, ins, outs = [], [], [], []
    for k in range(2):
        wq, wk = (1.0 + 0.1 * torch.randn(d, device="cuda")).half(), (1.0 + 0.1 * torch.randn(d, device="cuda")).half()
        bias = torch.randn(hq, 32, device="cuda").half()
        p = Z.WindowAttention(T, hq, hk, d, wq, wk, table, bias, STARTS["logs"], window=100, sinks=2)
        x = [torch.randn(T, h, d, device="cuda").half() for h in (hq, hk, hk, hq)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            p.forward(*x[:3])
            p.backward(x[3])
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = p.forward(*x[:3])
            grads = p.backward(x[3])
        places.append(p)
        graphs.append(g)
        ins.append(x)
        outs.append((o, *grads, *p.grads))
    eager = Z.WindowAttention(T, hq, hk, d, None, None, table, torch.zeros(hq, 32, device="cuda").half(), STARTS["logs"], window=100, sinks=2)
    for step in range(4):
        for k in (0, 1):
            for t in ins[k]:
                t.copy_(torch.randn_like(t))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for k in (0, 1):
            eager.wq, eager.wk, eager.bias = places[k].wq, places[k].wk, places[k].bias
            eager.dwq, eager.dwk = torch.zeros_like(eager.wq), torch.zeros_like(eager.wk)
            o = eager.forward(*ins[k][:3])
            want = (o, *eager.backward(ins[k][3]), *eager.grads)
            assert same(outs[k], want), (step, k)


def test_batches_without_tokens():
    p = Z.attention_params(4, 2, 64, starts=[0, 1])
    e = lambda h: torch.empty(0, h, 64, dtype=F16, device="cuda")
    bias = torch.ones(4, 2, dtype=F16, device="cuda")
    for kw in (dict(sequences=0), dict(sequences=3), dict(offsets=torch.zeros(1, dtype=torch.int32, device="cuda")),
               dict(offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))):
        Z.zero_attention_fwd(e(4), torch.empty(4, 0, device="cuda"), e(4), e(2), e(2), p, bias=bias, **kw)
        for accumulate, want in ((False, 0.0), (True, 7.0)):
            db = torch.full((4, 2), 7.0, device="cuda")
            Z.zero_attention_bwd(e(4), e(2), e(2), db, e(4), e(4), torch.empty(4, 0, device="cuda"), e(4), e(2), e(2), p, bias=bias,
                                 accumulate=accumulate, **kw)
            assert bool((db == want).all())
    for accumulate, want in ((False, 0.0), (True, 7.0)):
        dw = [torch.full((64,), 7.0, dtype=F16, device="cuda") for _ in range(2)]
        Z.zero_qk_norm_rope_fwd(e(4), e(2), e(4), e(2), None, None, None)
        Z.zero_qk_norm_rope_bwd(e(4), e(2), *dw, e(4), e(2), e(4), e(2), None, None, None, accumulate=accumulate)
        assert all(bool((t == want).all()) for t in dw)
    # tokens that no sequence has: the rows stay, the bias' gradient is 0
    c = Call([0, 0], 4, 2, 64, F16, starts=[0, 1], after=5)
    o, lse = c.fwd()
    assert bool((o == SENTINEL).all()) and bool((lse == SENTINEL).all())
    assert bool((c.bwd(o, lse)[3] == 0).all())


def test_offsets_out_of_order_stay_in_the_tensors():
    """Whatever the offsets hold, nothing outside the outputs' rows is written (the sentinels round them are checked)."""
    c = Call([100, 100], 2, 1, 64, F16, window=30, sinks=2, layout="odd", after=3)
    o, lse = c.fwd()
    for bad in ([0, 5, 2], [-7, 50, 10 ** 9], [200, 0, 100], [90, 30, 203], [2 ** 31 - 1, -2 ** 31, 0]):
        log("offsets", bad)
        c.where = {"offsets": torch.tensor(bad, dtype=torch.int32, device="cuda")}
        c.end = c.tokens
        c.fwd()
        c.bwd(o, lse)


def test_places_past_32_bits():
    """Tokens 2^23 elements apart: the last are past 2^32 elements, and 2^33 bytes, from the first."""
    T, h, d = 560, 2, 64
    buf = torch.zeros(T * (1 << 23) + 4096, dtype=F16, device="cuda")
    part = lambda k, n: torch.as_strided(buf, (T, n, d), (1 << 23, d, 1), 512 * k)
    c = Call([T - 60, 60], h, 1, d, F16, window=200, sinks=3)
    ins = {"q": part(0, h), "k": part(1, 1), "v": part(2, 1), "do": part(3, h)}
    o, lse = c.fwd()
    g = c.bwd(o, lse)
    for n, t in ins.items():
        t.copy_(c.d[n])
    c.d = ins
    o2, lse2 = part(4, h), torch.empty_like(lse)
    Z.zero_attention_fwd(o2, lse2, ins["q"], ins["k"], ins["v"], c.params, **c.where)
    outs = [part(5, h), part(6, 1), part(7, 1)]
    Z.zero_attention_bwd(*outs, None, ins["do"], o2, lse2, ins["q"], ins["k"], ins["v"], c.params, **c.where)
    assert torch.equal(o2, o) and torch.equal(lse2, lse) and same(outs, g[:3])
    table = torch.empty(T, d // 2, 2, device="cuda")
    Z.zero_rope_table(table)
    for interleaved in (False, True):
        y = [torch.empty_like(c.q, device="cuda"), torch.empty_like(c.k, device="cuda")]
        Z.zero_qk_norm_rope_fwd(*y, ins["q"].contiguous(), ins["k"].contiguous(), None, None, table, interleaved=interleaved)
        Z.zero_qk_norm_rope_fwd(outs[0], outs[1], ins["q"], ins["k"], None, None, table, interleaved=interleaved)
        assert same(outs[:2], y)


# ---- the place in a block ---------------------------------------------------------------------

class Place:
    """A place over a shard that holds its parameters (both norms' weights and the bias) at odd offsets."""

    def __init__(self, T, hq, hk, d, step, dtype=F16, **kw):
        g = torch.Generator().manual_seed(9)
        self.sizes = [d, d, hq * len(kw["starts"])]
        p = torch.cat([1.0 + 0.1 * torch.randn(2 * d, generator=g), 0.3 * torch.randn(self.sizes[2], generator=g)])
        step.p32[1:1 + len(p)].copy_(p)
        step.p32[0] = 0.0
        step.p16.copy_(step.p32.half())
        at = [1, 1 + d, 1 + 2 * d]
        self.views = [step.p16[a:a + n] for a, n in zip(at, self.sizes)]
        self.at = at
        self.table = torch.empty(T, d // 2, 2, device="cuda")
        Z.zero_rope_table(self.table)
        self.net = Z.WindowAttention(T, hq, hk, d, self.views[0], self.views[1], self.table, self.views[2].view(hq, -1), max_sequences=8, **kw)


def check_place(place, q, k, v, dout, o, grads, edges, positions, window, sinks, starts):
    """One forward and backward pass against the 64-bit forms, from the device's own stored values."""
    net = place.net
    cpu = lambda t: t.detach().cpu().double()
    T = q.shape[0]
    cs = A.angles(positions.cpu(), 64, 10000.0)
    for x, y, w in ((q, net._q[:T], net.wq), (k, net._k[:T], net.wk)):
        want, e = A.qk_fwd(cpu(x), cpu(w), cs, net.eps, False)
        top = (cpu(x) * (cpu(x).square().mean(2, keepdim=True) + net.eps).rsqrt() * cpu(w)).abs().amax(2, keepdim=True)
        close(y, want, A.stored(e + 2 * U * top, want, F16), "normed")
    nq, nk, vv, bias = cpu(net._q[:T]), cpu(net._k[:T]), cpu(v), cpu(net.bias)
    (wo, _), (eo, _) = A.attention_fwd(nq, nk, vv, bias, starts, net.params.scale, window, sinks, edges, F16)
    close(o, wo, A.stored(eo, wo, F16), "o")
    lse = cpu(net._lse[:net.params.heads * T].view(-1, T))
    (dq, dk, dv, db), (e_dq, e_dk, e_dv, e_db) = A.attention_bwd(cpu(dout), cpu(o), lse, nq, nk, vv, bias, starts, net.params.scale, window,
                                                               sinks, edges, F16)
    close(grads[2], dv, A.stored(e_dv, dv, F16), "dv")
    out = []
    for got, x, w, d1, e1 in ((grads[0], q, net.wq, dq, e_dq), (grads[1], k, net.wk, dk, e_dk)):
        # the gradient between the two passes is stored in binary16: its bound goes through the second one, which is linear in it
        e1 = A.stored(e1, d1, F16)
        x, w = cpu(x), cpu(w)
        (dx, dw), (e_dx, e_dw) = A.qk_bwd(d1, x, w, cs, net.eps, False)
        rstd = (x.square().mean(2, keepdim=True) + net.eps).rsqrt()
        h = (x * rstd).abs()
        one = A._spread(e1 + 2 * U * d1.abs().amax(2, keepdim=True), cs, False)
        gw = one * w.abs()
        e_dx = e_dx + rstd * (gw + h * (gw * h).mean(2, keepdim=True))
        close(got, dx, A.stored(e_dx, dx, F16), "dx")
        out.append((dw, e_dw + (one * h).sum((0, 1))))
    return out + [(db, e_db)]


def test_a_place_trained_through_the_shard_step():
    """Norms, rotation, windowed attention with bias, their backward passes, the flatten of the parameters' gradients, the decision and
    the update: two steps, the oracle's step bit for bit on the gradients that came out."""
    hq, hk, d, window, sinks = 4, 2, 64, 40, 2
    starts = Z.zero_attention_buckets(8, 30)
    lengths = [70, 1, 130]
    edges = [0, 70, 71, 201]
    T = edges[-1]
    n = 1 + 2 * d + hq * len(starts) + 2
    step = Z.ShardStep(n, fused=True)
    place = Place(T, hq, hk, d, step, starts=starts, window=window, sinks=sinks)
    net = place.net
    offsets = torch.tensor(edges, dtype=torch.int32, device="cuda")
    positions = torch.cat([torch.arange(m) for m in lengths]).int().cuda()
    segs = [(0, 0, 0, 1)] + [(i + 1, 0, a, m) for i, (a, m) in enumerate(zip(place.at, place.sizes))] + [(4, 0, n - 2, 2)]
    rest = [torch.zeros(1, dtype=F16, device="cuda"), torch.zeros(2, dtype=F16, device="cuda")]
    step.set_segments([rest[0], net.dwq, net.dwk, net.dbias.view(-1), rest[1]], segs)
    step.p32[n - 2:] = 0.0
    step.init_state(256.0)
    st_o, hp_o, hp = O.new_state(256.0), O.hparams(), Z.hparams()
    p32 = step.p32.cpu().numpy().copy()
    m, v32, p16 = np.zeros(n, np.float32), np.zeros(n, np.float32), p32.astype(np.float16).view(np.uint16)
    step.p16.copy_(torch.from_numpy(p16.view(np.float16)))
    g = torch.Generator().manual_seed(4)
    for k in range(2):
        log("step", k)
        qkv = torch.randn(T, (hq + 2 * hk) * d, generator=g).half().cuda()            # a joint projection's output
        part = lambda a, h: qkv[:, a * d:(a + h) * d].view(T, h, d)
        q, key, v = part(0, hq), part(hq, hk), part(hq + hk, hk)
        dqkv = torch.full_like(qkv, SENTINEL)
        dpart = lambda a, h: dqkv[:, a * d:(a + h) * d].view(T, h, d)
        dout = torch.randn(T, hq, d, generator=g).half().cuda()
        o = net.forward(q, key, v, offsets=offsets, positions=positions)
        grads = net.backward(dout, dpart(0, hq), dpart(hq, hk), dpart(hq + hk, hk))
        torch.cuda.synchronize()
        sums = check_place(place, q, key, v, dout, o, grads, edges, positions, window, sinks, starts)
        for got, (want, e) in zip(net.grads, sums):
            close(got, want, A.stored(e, want, F16), "parameters")
        srcs = [t.cpu().numpy().view(np.uint16).reshape(-1) for t in (rest[0], net.dwq, net.dwk, net.dbias, rest[1])]
        step.step(hp)
        grad_o = np.empty(n, np.uint16)
        O.step(hp_o, st_o, srcs, segs, grad_o, p16, p32, m, v32)
        torch.cuda.synchronize()
        s = step.read_state()
        assert (s.step, s.skip, s.sumsq) == (st_o.step, st_o.skip, st_o.sumsq) and s.skip == 0
        assert np.array_equal(step.grad16.cpu().numpy().view(np.uint16), grad_o)
        assert np.array_equal(step.p16.cpu().numpy().view(np.uint16), p16) and np.array_equal(step.p32.cpu().numpy(), p32)


def test_gradients_into_a_partition():
    """accumulate: two micro-batches' gradients added in an fp32 partition at odd places."""
    T, hq, hk, d = 150, 4, 4, 64
    starts = [0, 1, 5, 20]
    bias = torch.randn(hq, 4, device="cuda").half()
    net = Z.WindowAttention(T, hq, hk, d, torch.ones(d, device="cuda").half(), torch.ones(d, device="cuda").half(), None, bias, starts,
                            max_sequences=3)
    part = torch.zeros(3 + 2 * d + hq * 4, device="cuda")
    grads = [part[3:3 + d], part[3 + d:3 + 2 * d], part[3 + 2 * d:].view(hq, 4)]
    total = [torch.zeros_like(t) for t in grads]
    for k in range(2):
        x = [torch.randn(T, h, d, device="cuda").half() for h in (hq, hk, hk, hq)]
        net.forward(*x[:3], sequences=3)
        net.backward(x[3], grads=grads, accumulate=True)
        one = [torch.zeros_like(t) for t in grads]
        net.backward(x[3], grads=one)
        for t, n in zip(total, one):
            t += n
        # a backward pass without the parameters' gradients gives the same at the inputs
        assert same(net.backward(x[3], grads=(None, None, None)), net.backward(x[3]))
    assert same(grads, total) and bool((part[:3] == 0).all())


def test_place_takes_smaller_batches():
    """A place made for a batch that needs no parts of dk and dv, with batches that do."""
    place = Z.WindowAttention(8192, 64, 8, 128, window=256, sinks=4, max_sequences=4, dtype=BF16)
    g = torch.Generator(device="cuda").manual_seed(11)
    for tokens, n in ((8192, 4), (1024, 1), (384, 3), (1, 1), (2048, 2)):
        log("smaller", tokens, n)
        q, k, v, do = (torch.randn(tokens, h, 128, generator=g, device="cuda").to(BF16) for h in (64, 8, 8, 64))
        o = place.forward(q, k, v, sequences=n).clone()
        got = place.backward(do)
        alone = Z.WindowAttention(tokens, 64, 8, 128, window=256, sinks=4, max_sequences=n, dtype=BF16)
        assert torch.equal(alone.forward(q, k, v, sequences=n), o)
        assert same(alone.backward(do), got)


def test_place_with_rows_behind_the_last_sequence():
    """Rows in no sequence add nothing to the weights' gradients, whatever the gradients' memory held, and get 0."""
    heads, kv, dim, total, after = 6, 2, 64, 300, 37
    g = torch.Generator(device="cuda").manual_seed(3)
    wq, wk = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda") for _ in range(2))
    table = torch.empty(512, dim // 2, 2, device="cuda")
    Z.zero_rope_table(table)
    q, k, v, do = (torch.randn(total + after, h, dim, generator=g, device="cuda").half() for h in (heads, kv, kv, heads))
    offsets = torch.tensor([0, 100, 100, total], dtype=torch.int32, device="cuda")
    positions = torch.cat([torch.arange(100), torch.arange(200), torch.zeros(after)]).int().cuda()
    results = []
    for tokens in (total, total + after):
        place = Z.WindowAttention(total + after, heads, kv, dim, wq, wk, table, window=64, sinks=2, max_sequences=3, dtype=F16)
        place.forward(q[:tokens], k[:tokens], v[:tokens], offsets=offsets, positions=positions[:tokens])
        dq, dk, dv = (torch.full((tokens, h, dim), math.nan, dtype=F16, device="cuda") for h in (heads, kv, kv))
        dw = [torch.full((dim,), math.nan, device="cuda") for _ in range(2)]
        place.backward(do[:tokens], dq=dq, dk=dk, dv=dv, grads=(dw[0], dw[1], None))
        assert bool((dq[total:] == 0).all()) and bool((dk[total:] == 0).all()) and bool(dv[total:].isnan().all())
        results.append((dq[:total], dk[:total], dv[:total], dw))
    assert same(results[0][:3], results[1][:3])
    # The weights' gradients are binary32 sums of the same n addends (and zeros), in orders that may differ: two such sums are
    # at most 2 n 2^-24 times the sum of the addends' sizes apart.  An addend is an element of the attention's gradient, turned
    # back (at most its size and its partner's), times one of the normed head.
    nq, nk, o, lse = place._last[3:7]
    aq, ak, av = torch.zeros_like(nq), torch.zeros_like(nk), torch.empty_like(nk)
    Z.zero_attention_bwd(aq, ak, av, None, do, o, lse, nq, nk, v, place.params, offsets=offsets, sequences=3)
    for a, b, x, g2 in ((results[0][3][0], results[1][3][0], q, aq), (results[0][3][1], results[1][3][1], k, ak)):
        x, g2 = x[:total].double(), g2[:total].double().abs()
        h = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        sizes = ((g2 + g2.roll(dim // 2, -1)) * h.abs()).sum((0, 1))
        n = total * x.shape[1]
        assert bool(((a - b).abs().double() <= 2 * n * 2.0 ** -24 * sizes).all()) and bool(b.abs().max() > 0)


class WithoutBiasGradient(Call):
    def bwd(self, o, lse, grad_dtype=None, accumulate=False, start=0.0, workspace=None):
        outs = [self.out(h) for h in (self.hq, self.hk, self.hk)]
        Z.zero_attention_bwd(outs[0][1], outs[1][1], outs[2][1], None, self.d["do"], o, lse, self.d["q"], self.d["k"], self.d["v"], self.params,
                             bias=self.dbias, **self.where)
        return [v for _, v in outs] + [None]


@pytest.mark.parametrize("kind", [Call, WithoutBiasGradient])
@pytest.mark.parametrize("lengths,starts", [([1300], [0, 3, 601]), ([700, 500], [0, 3, 601]), ([300, 90], [0, 1, 5, 250])])
def test_bias_with_and_without_its_gradient(kind, lengths, starts):
    """Last buckets far out, in sequences that are long and short against them; the gradient wanted or not."""
    for dtype, dim in ((F16, 64), (BF16, 128)):
        log("bias gradient", kind.__name__, lengths, starts, dim)
        c = kind(lengths, 2, 1, dim, dtype, starts=starts, window=0, bias_dtype=F32)
        c.check_bwd(*c.check_fwd())
