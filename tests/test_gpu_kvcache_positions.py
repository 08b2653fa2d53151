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
