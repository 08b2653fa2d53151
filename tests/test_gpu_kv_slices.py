"""Attention with weights over more rows than scores are held for: the call goes over its
rows, and its sequences, in slices (needs a GPU). The tolerances are those of
test_gpu_kv.py; a slice adds its probabilities to the weights that the one before left, so each
of them rounds a weight once more (2^-24 of it)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lossless_bit_level_gb300 as ibp
from kv_harness import cache_of, offsets, pools, rounded
from test_gpu_kv import check_attention, run_attention

pytestmark = pytest.mark.gpu

SLICED = [
    # (lengths, query rows, q heads, kv heads, dim, page, code, table columns)
    ([300, 500], [300, 290], 4, 4, 64, 128, "int8", 1024),      # 512 rows fit: 256 of each sequence
    ([90, 0, 300, 33, 130], [40, 40, 40, 39, 1], 4, 2, 128, 128, "e4m3", 8192),  # 2 sequences at a time
    ([40, 70], [50, 70], 6, 2, 64, 16, "int8", 1 << 18),        # a group of three, more rows than tokens
    ([5, 20], [3, 2], 64, 1, 64, 128, "int8", 1 << 16),         # a row is 2 GiB: one at a time
]


@pytest.mark.parametrize("lens,counts,q_heads,heads,dim,page,code,cols", SLICED)
def test_rows_in_slices(lens, counts, q_heads, heads, dim, page, code, cols):
    rng = np.random.default_rng(sum(lens) + sum(counts))
    want = cache_of(rng, lens, heads, page, dim, code)
    cache = pools(want, rng, cols=cols)
    n = sum(counts)
    assert n * q_heads * cache.capacity * 4 > 1 << 30
    q = rounded(1.5 * rng.standard_normal((n, q_heads, dim)), "bf16").cuda()
    out, lse, w, w_in = run_attention(cache, q, counts, 0.125)
    check_attention(want, q, counts, 0.125, out, lse, w, w_in)
    again = run_attention(cache, q, counts, 0.125)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and torch.equal(w, again[2])


def test_a_prompt_with_weights_in_a_large_table():
    """The prompt of a sequence that may grow to 131,072 tokens, accumulated in place: what
    the cache class does before a first eviction."""
    rng = np.random.default_rng(2)
    n, heads, q_heads, dim, page = 700, 2, 8, 64, 64
    want = cache_of(rng, [n], heads, page, dim, "int8")
    cache = pools(want, rng, cols=2048)
    assert ibp.kv_attention_scratch_bytes(cache, n, n, q_heads, True) <= (1 << 30) + (64 << 20)
    q = rounded(rng.standard_normal((n, q_heads, dim)), "bf16").cuda()
    out, lse, w, w_in = run_attention(cache, q, [n], 0.125)
    check_attention(want, q, [n], 0.125, out, lse, w, w_in)
    acc = w_in.clone()
    scratch = torch.empty(ibp.kv_attention_scratch_bytes(cache, n, n, q_heads, True), dtype=torch.uint8, device="cuda")
    ibp.kv_attention(cache, q, torch.empty_like(q), 0.125, scratch, max_q=n, weights=acc,
                     weights_in=acc, decay=0.5)
    assert torch.equal(acc[0, :, :n], w[0, :, :n]) and torch.equal(acc[0, :, n:], w_in[0, :, n:])


@pytest.mark.parametrize("weights", [False, True])
def test_a_bound_far_above_the_rows_there_are(weights):
    """max_q as a program that captures graphs may set it: the same bits as with the exact one."""
    rng = np.random.default_rng(9)
    lens, counts = [300, 70, 5], [3, 1, 4]
    want = cache_of(rng, lens, 2, 16, 64, "int8")
    cache = pools(want, rng)
    q = rounded(rng.standard_normal((8, 4, 64)), "bf16").cuda()
    outs = []
    for max_q in (8, 1 << 20, 1 << 30):
        scratch = torch.empty(ibp.kv_attention_scratch_bytes(cache, 8, max_q, 4, weights),
                              dtype=torch.uint8, device="cuda")
        out, status = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
        w = torch.zeros((3, 2, cache.capacity), device="cuda") if weights else None
        ibp.kv_attention(cache, q, out, 0.125, scratch, cu_q=offsets(counts), max_q=max_q, weights=w,
                         status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        outs.append((out, w))
    for out, w in outs[1:]:
        assert torch.equal(out, outs[0][0]) and (w is None or torch.equal(w, outs[0][1]))
    check_attention(want, q, counts, 0.125, outs[0][0], None, None, None)
