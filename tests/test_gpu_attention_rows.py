"""Rows of a packed batch that are in no sequence."""
import math

import pytest
import torch

from test_gpu_attention import BF16, F16, F32, SENTINEL, strided, untouched

pytestmark = pytest.mark.gpu

import zero_partitioned_mixed_flatten_amd as Z  # noqa: E402


@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
def test_cleared(dtype):
    for layout in ("plain", "joint", "odd", "heads"):
        for dim in (8, 64, 80, 128):
            for edges in ([0, 0], [5, 9, 30], [0, 37], [37, 37], [0, 1, 36], [-3, 20], [0, 100], [30, 10]):
                buf, x = strided(37, 3, dim, dtype, layout)
                x.fill_(math.nan)
                Z.zero_attention_clear_rows(x, torch.tensor(edges, dtype=torch.int32, device="cuda"))
                first = min(max(edges[0], 0), 37)
                end = max(min(max(edges[-1], 0), 37), first)
                assert untouched(buf, x), (layout, dim, edges)
                assert bool((x[:first] == 0).all()) and bool((x[end:] == 0).all()) and bool(x[first:end].isnan().all())
    Z.zero_attention_clear_rows(torch.empty(0, 3, 64, dtype=dtype, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))


def test_cleared_on_another_stream():
    x = torch.full((300, 25, 64), math.nan, dtype=F16, device="cuda")
    offsets = torch.tensor([3, 3, 200], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Z.zero_attention_clear_rows(x, offsets, stream=s)
    s.synchronize()
    assert int(x.isnan().sum()) == 197 * 25 * 64


def test_cleared_past_32_bits():
    """Rows 2^24 elements apart: the last is past 2^32 elements."""
    buf = torch.full((300 << 24,), SENTINEL, dtype=F16, device="cuda")
    x = torch.as_strided(buf, (300, 2, 64), (1 << 24, 64, 1))
    Z.zero_attention_clear_rows(x, torch.tensor([1, 298], dtype=torch.int32, device="cuda"))
    assert bool((x[[0, 298, 299]] == 0).all()) and bool((x[1:298] == SENTINEL).all())
    assert bool((buf[299 << 24:][128:1 << 20] == SENTINEL).all())


def poison(shapes, dtype):
    """Leaves NaN in the memory that the next tensors of these shapes are likely to get."""
    ts = [torch.full(s, math.nan, dtype=dtype, device="cuda") for s in shapes]
    torch.cuda.synchronize()
    del ts


@pytest.mark.parametrize("before", [0, 11])
def test_a_place_and_rows_in_no_sequence(before):
    """Output and gradients that the place makes are 0 there, with whatever its memory held, after a longer batch too."""
    heads, kv, dim, total, after = 6, 2, 64, 300, 37
    tokens = before + total + after
    g = torch.Generator(device="cuda").manual_seed(4)
    wq, wk = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda") for _ in range(2))
    table = torch.empty(512, dim // 2, 2, device="cuda")
    Z.zero_rope_table(table)
    q, k, v, do = (torch.randn(tokens, h, dim, generator=g, device="cuda").half() for h in (heads, kv, kv, heads))
    place = Z.WindowAttention(tokens, heads, kv, dim, wq, wk, table, window=64, sinks=2, max_sequences=3, dtype=F16)
    positions = torch.cat([torch.zeros(before), torch.arange(100), torch.arange(200), torch.zeros(after)]).int().cuda()
    offsets = torch.tensor([before, before + 100, before + 100, before + total], dtype=torch.int32, device="cuda")
    everything = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    inside = slice(before, before + total)
    out = torch.ones(tokens, dtype=torch.bool, device="cuda")
    out[inside] = False
    place._o.fill_(math.nan)
    for longer in (False, True):
        if longer:
            place.forward(q, k, v, offsets=everything, positions=torch.arange(tokens, device="cuda").int())
        o = place.forward(q, k, v, offsets=offsets, positions=positions)
        assert bool((o[out] == 0).all()) and bool(o[inside].isfinite().all()) and bool((o[inside] != 0).any())
        poison([(tokens, heads, dim), (tokens, kv, dim), (tokens, kv, dim)], F16)
        dq, dk, dv = place.backward(do)
        for t in (dq, dk, dv):
            assert bool((t[out] == 0).all()) and bool(t[inside].isfinite().all())
    # given ones: o and dv stay as they are there
    o2 = torch.full_like(q, SENTINEL)
    place.forward(q, k, v, o=o2, offsets=offsets, positions=positions)
    assert bool((o2[out] == SENTINEL).all()) and torch.equal(o2[inside], o[inside])
    dv2 = torch.full_like(v, SENTINEL)
    got = place.backward(do, dv=dv2)
    assert got[2] is dv2 and bool((dv2[out] == SENTINEL).all()) and torch.equal(dv2[inside], dv[inside])
    assert torch.equal(got[0], dq) and torch.equal(got[1], dk)


def test_a_place_in_a_captured_graph():
    """Replays with other offsets in the same memory: each clears the rows that are outside now."""
    heads, kv, dim, tokens = 4, 2, 64, 200
    place = Z.WindowAttention(tokens, heads, kv, dim, max_sequences=2, dtype=F16)
    q, k, v, do = (torch.randn(tokens, h, dim, device="cuda").half() for h in (heads, kv, kv, heads))
    offsets = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        place.forward(q, k, v, offsets=offsets)
        place.backward(do)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = place.forward(q, k, v, offsets=offsets)
        grads = place.backward(do)
    other = Z.WindowAttention(tokens, heads, kv, dim, max_sequences=2, dtype=F16)
    for edges in ([0, 100, 150], [20, 30, 200], [0, 0, 7], [0, 100, 200]):
        offsets.copy_(torch.tensor(edges, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, *grads)]
        want = [other.forward(q, k, v, offsets=offsets), *other.backward(do)]
        for a, b in zip(got, want):
            assert torch.equal(a, b) and bool((a[:edges[0]] == 0).all()) and bool((a[edges[-1]:] == 0).all())
