"""Decoding loops over the 8-bit key/value cache with rotation on the way in, shared beginnings
and selected pages together, against the plain references (needs a GPU). Cached values are exact;
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
from test_gpu_kv_select import check_attention as check_selected, check_bounds, check_columns, select

pytestmark = pytest.mark.gpu


def append(cache, want, rng, counts, turns, rotation, heads, q_heads, dim):
    """A step's rows into both caches; the rotated queries, checked."""
    n = sum(counts)
    rows, q = random_rows(rng, n, heads, dim), rounded(rng.standard_normal((n, q_heads, dim)), "bf16")
    place = np.concatenate([np.arange(t, t + m) for t, m in zip(want.lens, counts)])[:, None]
    got = cache.append(rows["k"].cuda(), rows["v"].cuda(), counts, rotation=rotation, q=q.cuda())
    k = turn.rotated(rows["k"].float().numpy(), turns, place, [0] * (dim // 2), False)
    expected = torch.from_numpy(turn.rotated(q.float().numpy(), turns, place, [0] * (dim // 2), False)).bfloat16()
    assert torch.equal(got.cpu(), expected)
    at = 0
    for b, m in enumerate(counts):
        if m:
            want.append(b, {"k": k[at:at + m], "v": rows["v"][at:at + m].float().numpy()})
        at += m
    return got


def same_values(cache, want):
    k, v = cache.read(torch.float32)
    for name, got in (("k", k), ("v", v)):
        for b in range(want.batch):
            for h in range(want.heads):
                assert np.array_equal(got[b, :want.lens[b], h].cpu().numpy(), want.values(name, b, h)), (name, b, h)


@pytest.mark.parametrize("code,page,dim", [("int8", 16, 128), ("e4m3", 32, 64)])
def test_several_answers_to_one_prompt(code, page, dim):
    """One prompt, sequences that go on behind its shared pages, decoded for some steps."""
    heads, q_heads, batch = 2, 8, 6
    rng = np.random.default_rng(11)
    turns = turn.table(400, dim)
    rotation = ibp.KVRotation(torch.from_numpy(turns).cuda())
    cache = DecodeCache(n_pages=120, batch=batch, n_heads=heads, head_dim=dim, max_tokens=65_536, page_tokens=page,
                        code=code, track_weights=False)
    want = ref.Cache(batch, heads, page, dim, code)
    append(cache, want, rng, [150, 0, 0, 0, 0, 33], turns, rotation, heads, q_heads, dim)
    tokens = cache.share(0, [1, 2, 3])
    assert tokens == 150 // page * page
    for b in (1, 2, 3):
        for name in "kv":
            for h in range(heads):
                want.tiles[name][b][h] = [want.tiles[name][0][h][j] for j in range(tokens // page)]
        want.lens[b] = tokens
    scale = dim ** -0.5
    for step in range(6):
        counts = [[1] * 6, [1, 20, 3, 1, 2, 1]][step % 2]
        q = append(cache, want, rng, counts, turns, rotation, heads, q_heads, dim)
        n = sum(counts)
        lse = torch.empty((n, q_heads), device="cuda")
        out = cache.attend(q, scale, counts, lse=lse)
        check_attention(want, q, counts, scale, out, lse, None, None)
    same_values(cache, want)
    cache.check()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_decoding_over_selected_pages(code):
    """Rotated rows in, bounds kept up to date by every append, pages selected and attended."""
    heads, q_heads, dim, page, batch, pages = 2, 6, 64, 16, 3, 7
    rng = np.random.default_rng(12)
    turns = turn.table(500, dim)
    rotation = ibp.KVRotation(torch.from_numpy(turns).cuda())
    cache = DecodeCache(n_pages=100, batch=batch, n_heads=heads, head_dim=dim, max_tokens=480, page_tokens=page,
                        code=code, track_bounds=True)
    want = ref.Cache(batch, heads, page, dim, code)
    append(cache, want, rng, [333, 90, 200], turns, rotation, heads, q_heads, dim)
    for step in range(8):
        counts = [1, 1 + step % 3, 2]
        q = append(cache, want, rng, counts, turns, rotation, heads, q_heads, dim)
        check_bounds(want, cache.cache, cache.bounds, [0] * batch, 0)
        lse = torch.empty((sum(counts), q_heads), device="cuda")
        out = cache.attend(q, 0.125, counts, lse=lse, pages=pages)
        columns = select(cache.cache, cache.bounds, q, counts, pages)
        check_columns(want, q, counts, columns)
        check_selected(want, q, counts, 0.125, columns, out, lse)
    same_values(cache, want)
    # after an eviction the kept tokens' pages have bounds of their own
    cache.attend(q, 0.125, counts)
    cache.evict(100, 20)
    kept = ref.Cache(batch, heads, page, dim, code)
    k, v = cache.read(torch.float32)
    assert cache.lengths == [100, 100, 100]
    got, table = cache.bounds.cpu().numpy(), cache.cache.table.cpu().numpy()
    scales = cache.cache.k_scales.cpu().numpy()
    for b in range(batch):
        for j in range(-(-100 // page)):
            at = table[b, j]
            for h in range(heads):
                x = k[b, j * page:min(j * page + page, 100), h].cpu().numpy() / np.float32(scales[at, h])
                top = 127 if code == "int8" else 448
                lo, hi = np.floor(x.min(0) * 127 / top + 1e-3), np.ceil(x.max(0) * 127 / top - 1e-3)
                assert np.array_equal(got[at, h, 0], lo) and np.array_equal(got[at, h, 1], hi)
    lse = torch.empty((sum(counts), q_heads), device="cuda")
    out = cache.attend(q, 0.125, counts, lse=lse, pages=20)  # all pages: the same as a whole attention
    whole_lse = torch.empty_like(lse)
    whole = cache.attend(q, 0.125, counts, lse=whole_lse)
    assert bool(((out.float() - whole.float()).abs() <= 2.1 * 2.0 ** -8 * whole.float().abs() + 2.0 ** -18).all())
    assert bool(((lse - whole_lse).abs() <= 2.0 ** -18).all())
    cache.check()


def test_compressed_rows_are_rotated_on_the_way_in():
    """Rows kept losslessly compressed in host memory, rotated when they are loaded."""
    import ibp_inputs as gen
    from lossless_bit_level_gb300.offload import CompressedTensor
    heads, dim, n = 2, 128, 90
    dev = torch.device("cuda")
    words = [np.ascontiguousarray(gen.llm_kv(0, kv, n_rows=n)[:, :heads * dim]) for kv in (0, 1)]
    stores = [CompressedTensor.from_words(w, ibp.BF16, 0.9, 64, dev) for w in words]
    turns = turn.table(128, 64)
    cache = DecodeCache(n_pages=10, batch=1, n_heads=heads, head_dim=dim, max_tokens=128, page_tokens=32)
    cache.load(*stores, rotation=ibp.KVRotation(torch.from_numpy(turns).cuda(), interleaved=True))
    rows = [torch.from_numpy(w.view(np.int16).copy()).view(torch.bfloat16).view(n, heads, dim).float().numpy()
            for w in words]
    want = ref.Cache(1, heads, 32, dim, "int8")
    want.append(0, {"k": turn.rotated(rows[0], turns, np.arange(n)[:, None], [0] * 32, True), "v": rows[1]})
    same_values(cache, want)
    cache.check()
