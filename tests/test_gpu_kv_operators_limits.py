"""Attention behind shared beginnings and over selected pages where it goes wrong or far (needs a
GPU): bounded waits that run out (as in test_gpu_kv_timeout.py: the fetching warps stop after a
CTA's first tile, nothing faults), pools past 4 GB, two calls at once on two streams."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lossless_bit_level_gb300 as ibp
from kv_harness import offsets, pools, rounded
from test_gpu_kv import check_attention, status_word
from test_gpu_kv_select import attend, bounds_of, check_attention as check_selected, check_columns, select
from test_gpu_kv_shared import run_shared, shared_cache

pytestmark = pytest.mark.gpu


def long_cache(dim, batch=6, heads=8, page=64, tokens=12_000, own=3_000, seed=0):
    """Random codes; every sequence's first `tokens` are those of sequence 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shared, mine = -(-tokens // page), -(-own // page)
    shape = (shared + batch * mine, heads, page, dim)
    k, v = (torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand(shape[:2], generator=g, device="cuda") * 0.01 for _ in range(2))
    table = torch.cat([torch.arange(shared).expand(batch, -1),
                       shared + torch.arange(batch * mine).view(batch, mine)], 1).to(torch.int32)
    lens = torch.full((batch,), shared * page + own, dtype=torch.int32, device="cuda")
    return ibp.KVCache(k, v, ks, vs, table.cuda().contiguous(), lens), shared * page


def runs_out(call):
    """A call whose waits run out records that, and the next gives the bits of the one before."""
    before = call()
    assert before[0] == 0 and bool(torch.isfinite(before[1].float()).all())
    limit, held = ibp.testing_set_wait_limit_ns(1_000_000), ibp.testing_withhold_plans(True)
    try:
        assert call()[0] == ibp.ERR_TIMEOUT
    finally:
        ibp.testing_withhold_plans(held)
        ibp.testing_set_wait_limit_ns(limit)
    after = call()
    assert after[0] == 0 and torch.equal(before[1], after[1])


@pytest.mark.parametrize("q_heads,n,dim", [(8, 1, 128), (64, 1, 128), (64, 4, 64)])
def test_shared_waits_run_out_then_the_stream_recovers(q_heads, n, dim):
    """6 rows a head (the kernel for few alone), 48 (both halves of the one for many), 192."""
    cache, prefix = long_cache(dim)
    q = rounded(np.random.default_rng(n).standard_normal((6 * n, q_heads, dim)), "bf16").cuda()
    scratch = torch.zeros(ibp.kv_attention_shared_scratch_bytes(cache, 6 * n, n, q_heads, 1, 6 * n),
                          dtype=torch.uint8, device="cuda")
    groups, tokens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 6], [prefix]))
    stream = torch.cuda.Stream()

    def call():
        status, out = status_word(), torch.zeros_like(q)
        stream.wait_stream(torch.cuda.current_stream())
        ibp.kv_attention_shared(cache, q, out, 0.1, scratch, groups, tokens, 6 * n, max_q=n, status=status,
                                stream=stream)
        stream.synchronize()
        return int(status.item()), out

    runs_out(call)


@pytest.mark.parametrize("n,dim", [(1, 128), (3, 64)])
def test_selected_waits_run_out_then_the_stream_recovers(n, dim):
    cache, _ = long_cache(dim)
    bounds = bounds_of(cache)
    ibp.kv_bounds(cache, bounds)
    q = rounded(np.random.default_rng(n).standard_normal((6 * n, 16, dim)), "bf16").cuda()
    columns = select(cache, bounds, q, [n] * 6, 200)

    def call():
        status = status_word()
        out, _ = attend(cache, columns, q, [n] * 6, 0.1, status=status)
        torch.cuda.synchronize()
        return int(status.item()), out

    runs_out(call)


@pytest.mark.parametrize("many", [False, True])
def test_two_calls_at_once(many):
    """Shared and selected calls on two streams, each with its own workspace."""
    rng = np.random.default_rng(3)
    groups = [(600, [40, 70, 9] * (5 if many else 1))]
    counts = [1] * len(groups[0][1])
    scale, work = 0.125, []
    for code in ("int8", "e4m3"):
        want, cache = shared_cache(rng, groups, 2, 16, 64, code)
        bounds = bounds_of(cache)
        ibp.kv_bounds(cache, bounds)
        work.append((want, cache, bounds, rounded(rng.standard_normal((len(counts), 8, 64)), "bf16").cuda()))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    n = len(counts)
    buffers = [(torch.empty(1 << 27, dtype=torch.uint8, device="cuda"), torch.empty_like(w[3]),
                torch.empty((n, 8), device="cuda"), torch.empty((n, 2, 9), dtype=torch.int32, device="cuda"),
                torch.empty_like(w[3]), torch.empty((n, 8), device="cuda"),
                torch.empty(1 << 24, dtype=torch.uint8, device="cuda")) for w in work]
    starts, prefix = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [600]))
    torch.cuda.synchronize()
    for _ in range(20):
        for (_, cache, bounds, q), (scratch, out, lse, columns, chosen, chosen_lse, small), stream in zip(
                work, buffers, streams):
            ibp.kv_attention_shared(cache, q, out, scale, scratch, starts, prefix, n, lse=lse, stream=stream)
            ibp.kv_select(cache, bounds, q, columns, small, stream=stream)
            ibp.kv_attention_selected(cache, columns, q, chosen, scale, small, lse=chosen_lse, stream=stream)
    torch.cuda.synchronize()
    for (want, _, _, q), (_, out, lse, columns, chosen, chosen_lse, _) in zip(work, buffers):
        check_attention(want, q, counts, scale, out, lse, None, None)
        check_columns(want, q, counts, columns)
        check_selected(want, q, counts, scale, columns, chosen, chosen_lse)


def test_pages_past_four_gigabytes():
    """The last pages of a pool of 4.8 GB: rotated append, bounds, selection and both attentions."""
    heads, page, dim, n_pages = 8, 128, 128, 37_000
    rng = np.random.default_rng(4)
    small_groups = [(256, [150, 300])]
    want, small = shared_cache(rng, small_groups, heads, page, dim, "int8")
    room = torch.empty((n_pages, heads, page, dim), dtype=torch.int8, device="cuda")
    scales = torch.full((2, n_pages, heads), float("nan"), device="cuda")
    first = n_pages - small.k_codes.shape[0]
    v = torch.empty_like(room)
    room[first:], v[first:] = small.k_codes, small.v_codes
    scales[0, first:], scales[1, first:] = small.k_scales, small.v_scales
    table = torch.where(small.table >= 0, small.table + first, small.table)
    cache = ibp.KVCache(room, v, scales[0], scales[1], table.contiguous(), small.lens)
    bounds = torch.empty((n_pages, heads, 2, dim), dtype=torch.int8, device="cuda")
    status = status_word()
    ibp.kv_bounds(cache, bounds, status=status)
    q = rounded(rng.standard_normal((2, 16, dim)), "bf16").cuda()
    columns = select(cache, bounds, q, [1, 1], 3, status=status)
    check_columns(want, q, [1, 1], columns)
    out, lse = attend(cache, columns, q, [1, 1], 0.09, status=status)
    check_selected(want, q, [1, 1], 0.09, columns, out, lse)
    out, lse = run_shared(cache, small_groups, q, [1, 1], 0.09)
    check_attention(want, q, [1, 1], 0.09, out, lse, None, None)
    rotation = ibp.KVRotation(ibp.rotation_table(600, dim))
    k = rounded(rng.standard_normal((2, heads, dim)), "bf16").cuda()
    new_lens = torch.empty_like(cache.lens)
    ibp.kv_append_rotated(cache, k, k, rotation, new_lens=new_lens, status=status, cu=offsets([1, 1]))
    got = torch.empty((2, 1, heads, dim), device="cuda")
    after = ibp.KVCache(room, v, scales[0], scales[1], cache.table, new_lens)
    ibp.kv_read(after, None, got, begin=cache.lens, status=status)
    assert int(status.item()) == 0
    half = scales[1][table.gather(1, (cache.lens // page).long()[:, None])[:, 0].long()][:, None, :, None] / 2
    # a code is off by half a unit of its page's scale at most (and the product's rounding)
    assert bool(((got - k.float()[:, None]).abs() <= half * (1 + 2.0 ** -20)).all())
