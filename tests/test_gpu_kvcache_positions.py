"""Decoding with rotated rows before and after evictions (needs a GPU): kept keys stay rotated by
their own numbers and new ones go on behind them. Cached values and rotated queries are exact;
attention's tolerances are those of test_gpu_kv.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
import kv_rotate_reference as turn
import lossless_bit_level_gb300 as ibp
from kv_harness import random_rows, rounded
from lossless_bit_level_gb300.kvcache import DecodeCache
from test_gpu_kv import check_attention
from test_gpu_kv_select import check_attention as check_selected, check_columns, select
from test_gpu_kvcache_operators import same_values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("axes,code,dim", [(1, "int8", 128), (3, "e4m3", 64)])
def test_rotation_after_an_eviction(axes, code, dim):
    heads, q_heads, batch, page = 2, 6, 4, 16
    rng = np.random.default_rng(axes)
    turns, axis = turn.table(600, dim), [i % axes for i in range(dim // 2)]
    rotation = ibp.KVRotation(torch.from_numpy(turns).cuda(), axis=axis)
    cache = DecodeCache(n_pages=160, batch=batch, n_heads=heads, head_dim=dim, max_tokens=480, page_tokens=page,
                        code=code)
    want, seen = ref.Cache(batch, heads, page, dim, code), np.zeros(batch, int)
    scale = dim ** -0.5

    def step(counts, own=None):
        nonlocal seen
        n = sum(counts)
        rows, q = random_rows(rng, n, heads, dim), rounded(rng.standard_normal((n, q_heads, dim)), "bf16")
        numbers = np.concatenate([np.arange(t, t + m) for t, m in zip(seen, counts)])
        place = np.repeat(numbers[:, None], axes, 1) if own is None else own
        got = cache.append(rows["k"].cuda(), rows["v"].cuda(), counts, rotation=rotation, q=q.cuda(),
                           positions=None if own is None else torch.from_numpy(own.astype(np.int32)).cuda())
        expected = turn.rotated(q.float().numpy(), turns, place, axis, False)
        assert torch.equal(got.cpu(), torch.from_numpy(expected).bfloat16())
        k, at = turn.rotated(rows["k"].float().numpy(), turns, place, axis, False), 0
        for b, m in enumerate(counts):
            if m:
                want.append(b, {"k": k[at:at + m], "v": rows["v"][at:at + m].float().numpy()})
            at += m
        seen = seen + counts
        lse = torch.empty((n, q_heads), device="cuda")
        out = cache.attend(got, scale, counts, lse=lse)
        check_attention(want, got, counts, scale, out, lse, None, None)
        same_values(cache, want)

    step([333, 90, 0, 40])
    for budget, recent in ((100, 20), (60, 60), (48, 0)):
        weights = cache.weights.cpu().numpy()
        want, _ = want.evict([[w[:n] for w in of_one] for of_one, n in zip(weights, want.lens)], budget, recent)
        cache.evict(budget, recent)
        assert cache.lengths == want.lens
        same_values(cache, want)
        step([1, 17, 3, 2])
        step([2, 1, 1, 30])
    step([1, 1, 1, 1], own=rng.integers(0, 600, (4, axes)))
    step([1, 1, 1, 1])
    cache.check()


@pytest.mark.parametrize("code,page,dim", [("int8", 16, 64), ("e4m3", 32, 128)])
def test_sharing_what_an_eviction_left(code, page, dim):
    """Sequences that begin with the kept pages of an evicted one, go on with numbers behind all of
    them, and attend over a few of their pages."""
    heads, q_heads, batch, pages = 2, 4, 4, 5
    rng = np.random.default_rng(page)
    turns = turn.table(500, dim)
    rotation = ibp.KVRotation(torch.from_numpy(turns).cuda())
    cache = DecodeCache(n_pages=90, batch=batch, n_heads=heads, head_dim=dim, max_tokens=480, page_tokens=page,
                        code=code, track_bounds=True)
    want, scale = ref.Cache(batch, heads, page, dim, code), dim ** -0.5

    def step(counts, numbers):
        n = sum(counts)
        rows, q = random_rows(rng, n, heads, dim), rounded(rng.standard_normal((n, q_heads, dim)), "bf16")
        place = np.concatenate([np.arange(t, t + m) for t, m in zip(numbers, counts)])[:, None]
        got = cache.append(rows["k"].cuda(), rows["v"].cuda(), counts, rotation=rotation, q=q.cuda())
        expected = turn.rotated(q.float().numpy(), turns, place, [0] * (dim // 2), False)
        assert torch.equal(got.cpu(), torch.from_numpy(expected).bfloat16())
        k, at = turn.rotated(rows["k"].float().numpy(), turns, place, [0] * (dim // 2), False), 0
        for b, m in enumerate(counts):
            if m:
                want.append(b, {"k": k[at:at + m], "v": rows["v"][at:at + m].float().numpy()})
            at += m
        lse = torch.empty((n, q_heads), device="cuda")
        out = cache.attend(got, scale, counts, lse=lse)
        check_attention(want, got, counts, scale, out, lse, None, None)
        return got

    step([333, 0, 0, 25], [0, 0, 0, 0])
    weights = cache.weights.cpu().numpy()
    want, kept = want.evict([[w[:n] for w in of_one] for of_one, n in zip(weights, want.lens)], 200, 30)
    cache.evict(200, 30)
    tokens = cache.share(0, [1, 2])
    assert tokens == 192
    numbers = [333, 333 - 8, 333 - 8, 25]
    for h in range(heads):
        assert kept[0][h][tokens - 1] < numbers[1]  # no shared token has a number from there on
        for b in (1, 2):
            for name in "kv":
                want.tiles[name][b][h] = list(want.tiles[name][0][h][:tokens // page])
    want.lens[1] = want.lens[2] = tokens
    for counts in ([1, 1, 1, 1], [1, 20, 3, 1], [2, 1, 1, 40]):
        got = step(counts, numbers)
        numbers = [a + b for a, b in zip(numbers, counts)]
        lse = torch.empty((sum(counts), q_heads), device="cuda")
        out = cache.attend(got, scale, counts, lse=lse, pages=pages)
        columns = select(cache.cache, cache.bounds, got, counts, pages)
        check_columns(want, got, counts, columns)
        check_selected(want, got, counts, scale, columns, out, lse)
    same_values(cache, want)
    cache.check()
