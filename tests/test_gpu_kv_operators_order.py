"""Kernels that start while the one before them ends read nothing of it before it is there (needs a
GPU): selection, attention over selected pages and behind shared beginnings right behind a kernel
that writes their inputs for a long time, as plain calls and as nodes of a graph, and what comes
behind them in the stream."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lossless_bit_level_gb300 as ibp
from kv_harness import rounded
from test_gpu_kv_select import bounds_of
from test_gpu_kv_shared import shared_cache

pytestmark = pytest.mark.gpu


def step(cache, source, q, slow, outs, scratch, groups, prefix):
    """The queries arrive at the end of a long kernel (an index over many rows), then the calls, then
    a copy of what they wrote."""
    torch.index_select(source.view(-1, 64), 0, slow, out=q.view(-1, 64))
    n = q.shape[0]
    columns, chosen, out = outs[:3]
    ibp.kv_select(cache, outs[3], q, columns, scratch)
    ibp.kv_attention_selected(cache, columns, q, chosen, 0.125, scratch)
    ibp.kv_attention_shared(cache, q, out, 0.125, scratch, groups, prefix, n)
    outs[4].copy_(columns)
    outs[5].copy_(chosen)
    outs[6].copy_(out)


@pytest.mark.parametrize("answers", [3, 40])  # few rows, and rows for the kernel for many
@pytest.mark.parametrize("graph", [False, True])
def test_right_behind_a_kernel_that_writes_their_inputs(answers, graph):
    rng = np.random.default_rng(answers)
    heads, q_heads = 2, 8
    want, cache = shared_cache(rng, [(400, [int(t) for t in rng.integers(0, 90, answers)])], heads, 16, 64, "int8")
    bounds = bounds_of(cache)
    ibp.kv_bounds(cache, bounds)
    rows = answers * q_heads
    sources = [rounded(rng.standard_normal((answers, q_heads, 64)), "bf16").cuda() for _ in range(2)]
    q, slow = torch.empty_like(sources[0]), torch.arange(rows, device="cuda")
    outs = [torch.empty((answers, heads, 6), dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty_like(q),
            bounds, torch.empty((answers, heads, 6), dtype=torch.int32, device="cuda"), torch.empty_like(q),
            torch.empty_like(q)]
    scratch = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    groups, prefix = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, answers], [400]))
    heavy = torch.randn((4096, 4096), device="cuda")
    args = (q, slow, outs, scratch, groups, prefix)
    expected = []
    for source in sources:  # waited for after every call
        step(cache, source, *args)
        torch.cuda.synchronize()
        expected.append([t.clone() for t in outs[4:]])
    assert not torch.equal(expected[0][2], expected[1][2])
    replays = []
    if graph:
        for source in sources:
            stream = torch.cuda.Stream()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                step(cache, source, *args)
            replays.append(g)
    for i in range(40):
        torch.mm(heavy, heavy, out=heavy.new_empty(heavy.shape))  # the stream is behind the host
        if graph:
            replays[i % 2].replay()
        else:
            step(cache, sources[i % 2], *args)
        got = [t.clone() for t in outs[4:]]
        for a, b in zip(got, expected[i % 2]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("q_rows", [False, True])  # queries in a launch of their own behind the keys
def test_selection_right_behind_an_append_that_raises_scales(q_rows):
    batch, heads, d, page, old, new = 24, 32, 128, 32, 20, 40
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rows(n, times):
        return (times * torch.randn((n, heads, d), generator=gen, device="cuda")).to(torch.bfloat16)

    n_pages = 2 * batch
    codes = [torch.zeros((n_pages, heads, page, d), dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((n_pages, heads), device="cuda") for _ in range(2)]
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").view(batch, 2)
    lens = [torch.full((batch,), n, dtype=torch.int32, device="cuda") for n in (0, old, old + new)]
    caches = [ibp.KVCache(*codes, *scales, table, x) for x in lens]
    turn = ibp.KVRotation(ibp.rotation_table(old + new, d))
    ibp.kv_append(caches[0], rows(batch * old, 1.0), rows(batch * old, 1.0))
    start = [t.clone() for t in (*codes, *scales)]
    k, v, wide = rows(batch * new, 30.0), rows(batch * new, 30.0), rows(batch * new, 1.0)
    turned = torch.empty_like(wide) if q_rows else None  # (its launch comes between)
    q, out = rows(batch, 1.0), torch.empty((batch, heads, d), dtype=torch.bfloat16, device="cuda")
    bounds = torch.zeros(caches[0].bounds_shape, dtype=torch.int8, device="cuda")
    columns = torch.empty((batch, heads, 2), dtype=torch.int32, device="cuda")
    one = torch.zeros((batch, heads, 2), dtype=torch.int32, device="cuda") + torch.arange(2, device="cuda").int()
    scratch = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")

    def run(wait):
        for t, x in zip((*codes, *scales), start):
            t.copy_(x)
        ibp.kv_append_rotated(caches[1], k, v, turn, q=wide if q_rows else None, q_out=turned)
        if wait:
            torch.cuda.synchronize()
        ibp.kv_attention_selected(caches[2], one, q, out, 0.1, scratch)
        if wait:
            torch.cuda.synchronize()
        ibp.kv_bounds(caches[2], bounds)
        ibp.kv_select(caches[2], bounds, q, columns, scratch)
        return [t.clone() for t in (out, columns, bounds, *scales)]

    expected = run(True)
    assert (scales[0] > start[2]).any()
    heavy = torch.randn((4096, 4096), device="cuda")
    for i in range(20):
        torch.mm(heavy, heavy, out=heavy.new_empty(heavy.shape))
        for a, b in zip(run(False), expected):
            assert torch.equal(a, b), i
