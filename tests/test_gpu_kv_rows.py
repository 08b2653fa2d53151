"""Attention of many query rows over the 8-bit cache (the matrix-unit path: more than 32
rows of a K/V head, no weights), where its own arithmetic can go wrong (needs a GPU). The
tolerances are those of test_gpu_kv.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
import lossless_bit_level_gb300 as ibp
from kv_harness import cache_of, offsets, pools, rounded, with_lens
from test_gpu_kv import check_attention, run_attention, status_word

pytestmark = pytest.mark.gpu

ROWS = [
    # (lengths, query rows, q heads, kv heads, dim, page, code, dtype)
    ([50], [33], 1, 1, 128, 16, "int8", "fp16"),
    ([128], [65], 1, 1, 128, 128, "int8", "bf16"),
    ([129], [129], 1, 1, 64, 16, "e4m3", "fp16"),
    ([255, 257, 0, 1, 640], [255, 100, 90, 1, 3], 4, 2, 128, 64, "int8", "bf16"),
    ([40, 300], [200, 90], 5, 1, 64, 32, "int8", "fp16"),        # more queries than tokens
    ([1000, 77], [10, 77], 24, 2, 128, 16, "e4m3", "bf16"),      # twelve heads to a key head
    ([1500], [1100], 3, 3, 128, 64, "int8", "fp16"),
    ([2000, 3, 500], [70, 3, 500], 2, 2, 64, 128, "e4m3", "bf16"),
    ([30, 0, 700, 2], [600, 300, 40, 530], 3, 3, 64, 16, "int8", "bf16"),  # blocks that see nothing
]


@pytest.mark.parametrize("lens,counts,q_heads,heads,dim,page,code,dtype", ROWS)
def test_many_rows(lens, counts, q_heads, heads, dim, page, code, dtype):
    rng = np.random.default_rng(sum(lens) + 3 * sum(counts) + q_heads)
    want = cache_of(rng, lens, heads, page, dim, code)
    cache = pools(want, rng)
    q = rounded(1.5 * rng.standard_normal((sum(counts), q_heads, dim)), dtype).cuda()
    scale = 1.0 / np.sqrt(dim)
    out, lse, _, _ = run_attention(cache, q, counts, scale, weights=False)
    check_attention(want, q, counts, scale, out, lse, None, None)
    for _ in range(3):
        again = run_attention(cache, q, counts, scale, weights=False)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("page", [16, 64])
def test_growing_scores_and_far_value_scales(page, weights):
    """Scores that rise along the sequence (references are raised again and again, by little
    and by much), value scales far apart from page to page, pages of zeros; a negative and a
    zero scale; by both kernels (the one for few rows takes all calls with weights).

    Where one token holds nearly all of a row's output but has a zero there, the element
    comes from factors far below the largest. fp16 holds a factor to 2^-25, the largest
    factor is 2^2 or more, so each of T tokens may be off by 2^-27 of the largest p_t times
    its page's value scale, times a code (127)."""
    rng = np.random.default_rng(page)
    dim, n, total = 64, 130, 512
    want = ref.Cache(1, 1, page, dim, "int8")
    factors = [1.0, 1e-12, 1e15, 0.0, 3.0, 1e-25, 1e4, 0.5]
    for j in range(total // page):
        k = rng.standard_normal((page, 1, dim)).astype(np.float32) * (0.2 + 12.0 * j * page / total)
        v = rng.standard_normal((page, 1, dim)).astype(np.float32) * factors[j % 8]
        want.append(0, {"k": k, "v": v.astype(np.float32)})
    cache = pools(want, rng)
    scales = np.repeat([s for s, _ in want.tiles["v"][0][0]], page).astype(np.float64)
    for scale, gain in ((0.125, 2.0), (1.0, 1.0), (-0.25, 1.5), (0.0, 1.0)):
        q = rounded(gain * rng.standard_normal((n, 1, dim)), "bf16").cuda()
        out, lse, _, _ = run_attention(cache, q, [n], scale, weights=weights)
        k, v = want.values("k", 0, 0), want.values("v", 0, 0)
        qn = q.float().cpu().numpy()
        o, z, _ = ref.attention(qn, k, v, scale)
        size, _, _ = ref.attention(qn, k, np.abs(v), scale)
        x = scale * (qn.reshape(n, dim).astype(np.float64) @ k.T.astype(np.float64)) - z
        x = np.where(np.arange(total) < total - n + 1 + np.arange(n)[:, None], x, -np.inf)
        largest = (np.exp(x) * scales).max(1)[:, None, None]
        spread = abs(scale) * (np.abs(qn).reshape(n, dim) @ np.abs(k).T).max()
        score = 2.0 ** -20 * spread + 2.0 ** -21
        tol = 2.0 ** -8 * 1.01 * np.abs(o) + (2.0 ** -11 + 2 * score) * size + 2.0 ** -24 + \
            total * 2.0 ** -27 * 127 * largest
        assert (np.abs(out.float().cpu().numpy() - o) <= tol).all()
        assert (np.abs(lse.cpu().numpy() - z) <= score + 2.0 ** -22 * np.abs(z)).all()


def test_many_rows_strides_and_missing_pages():
    """Views of fused tensors; a page that is not there is reported and not attended."""
    rng = np.random.default_rng(3)
    lens, n, dim, page = [300], 100, 128, 64
    want = cache_of(rng, lens, 2, page, dim, "int8")
    cache = pools(want, rng)
    fused = rounded(rng.standard_normal((n, 9, dim)), "bf16").cuda()
    q = fused[:, 1:9:2]
    out = torch.zeros((n, 10, dim), dtype=torch.bfloat16, device="cuda")
    got, lse, _, _ = run_attention(cache, q, [n], 0.08, weights=False, out=out[:, 3:7])
    check_attention(want, q, [n], 0.08, got, lse, None, None)
    assert not out[:, :3].any() and not out[:, 7:].any()
    cache.table[0, 1] = -5
    status = status_word()
    scratch = torch.empty(ibp.kv_attention_scratch_bytes(cache, n, n, 4, False), dtype=torch.uint8,
                          device="cuda")
    o = torch.empty((n, 4, dim), dtype=torch.bfloat16, device="cuda")
    ibp.kv_attention(cache, q, o, 0.08, scratch, cu_q=offsets([n]), max_q=n, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == ibp.ERR_INDEX
    for h in range(2):
        k, v = want.values("k", 0, h), want.values("v", 0, h)
        mine = q[:, 2 * h:2 * h + 2].float().cpu().numpy()
        for i in (0, n - 1):
            seen = np.array([t for t in range(300 - n + i + 1) if not 64 <= t < 128])
            x, _, _ = ref.attention(mine[i:i + 1], k[seen], v[seen], 0.08)
            assert np.abs(o[i, 2 * h:2 * h + 2].float().cpu().numpy() - x[0]).max() <= 2.0 ** -7


@pytest.mark.parametrize("n", [1, 40])
def test_more_sequences_than_one_launch_takes(n):
    """600 sequences: several launches, for few rows and for many."""
    rng = np.random.default_rng(n)
    batch, group, dim, page = 600, 2, 64, 16
    lens = [int(x) for x in rng.integers(0, 60, batch)]
    want = cache_of(rng, lens, 1, page, dim, "int8")
    cache = pools(want, rng)
    counts = [n] * batch
    q = rounded(rng.standard_normal((batch * n, group, dim)), "bf16").cuda()
    out, lse, w, w_in = run_attention(cache, q, counts, 0.125, weights=n == 1, cu=n > 1)
    check_attention(want, q, counts, 0.125, out, lse, w, w_in)


def test_many_rows_graph_and_lengths_changed_between_replays():
    rng = np.random.default_rng(8)
    want = cache_of(rng, [400], 1, 64, 128, "e4m3")
    cache = pools(want, rng)
    lens = cache.lens.clone()
    view = with_lens(cache, lens)
    q = rounded(rng.standard_normal((90, 1, 128)), "fp16").cuda()
    out, status = torch.empty_like(q), status_word()
    scratch = torch.empty(ibp.kv_attention_scratch_bytes(view, 90, 90, 1, False), dtype=torch.uint8,
                          device="cuda")
    ibp.kv_attention(view, q, out, 0.09, scratch, max_q=90, status=status)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ibp.kv_attention(view, q, out, 0.09, scratch, max_q=90, status=status)
    qn = q.float().cpu().numpy()
    for t in (400, 90, 33, 0, 399):
        lens.fill_(t)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        k, v = want.values("k", 0, 0, t), want.values("v", 0, 0, t)
        o, _, _ = ref.attention(qn, k, v, 0.09)
        size, _, _ = ref.attention(qn, k, np.abs(v), 0.09)
        tol = 2.0 ** -11 * 1.01 * np.abs(o) + 2.0 ** -10 * size + 2.0 ** -24
        assert (np.abs(out.float().cpu().numpy() - o) <= tol).all()
    assert int(status.item()) == 0
