"""A decoding loop over the 8-bit key/value cache, together with the codec (needs a GPU):
rows kept losslessly compressed in host memory are loaded, tokens are appended and attended
one by one, the cache is cut to a budget, and everything is compared with the plain
reference; what is read back goes through the codec again."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ibp_inputs as gen
import kv_reference as ref
import lossless_bit_level_gb300 as ibp
from kv_harness import random_rows
from lossless_bit_level_gb300.kvcache import DecodeCache
from lossless_bit_level_gb300.offload import CompressedTensor

pytestmark = pytest.mark.gpu


def bf16_rows(words: np.ndarray, heads: int) -> torch.Tensor:
    return torch.from_numpy(words.view(np.int16).copy()).view(torch.bfloat16).view(
        words.shape[0], heads, -1)


@pytest.mark.parametrize("code,page", [("int8", 16), ("e4m3", 64)])
def test_decoding_loop(code, page):
    heads, dim, q_heads, batch, prompt = 4, 128, 8, 3, 100
    dev, rng = torch.device("cuda"), np.random.default_rng(7)
    words = [np.ascontiguousarray(gen.llm_kv(0, kv, n_rows=batch * prompt)[:, :heads * dim])
             for kv in (0, 1)]
    stores = [CompressedTensor.from_words(w, ibp.BF16, 0.9, 64, dev) for w in words]
    cache = DecodeCache(n_pages=60, batch=batch, n_heads=heads, head_dim=dim, max_tokens=200,
                        page_tokens=page, code=code, decay=0.9)
    counts = [100, 150, 50]
    cache.load(*stores, counts=counts)
    want = ref.Cache(batch, heads, page, dim, code)
    prompt_rows = [bf16_rows(w, heads).float().numpy() for w in words]
    at = 0
    for b, n in enumerate(counts):
        want.append(b, {"k": prompt_rows[0][at:at + n], "v": prompt_rows[1][at:at + n]})
        at += n
    weights = [[np.zeros(n) for _ in range(heads)] for n in counts]
    budget, recent = 90, 20
    for step in range(12):
        rows = random_rows(rng, batch, heads, dim)
        cache.append(rows["k"].cuda(), rows["v"].cuda())
        q = torch.from_numpy(rng.standard_normal((batch, q_heads, dim)).astype(np.float32)).bfloat16()
        out = cache.attend(q.cuda(), dim ** -0.5).float().cpu().numpy()
        got = cache.weights.cpu().numpy()
        for b in range(batch):
            want.append(b, {n: t[b:b + 1].float().numpy() for n, t in rows.items()})
            for h in range(heads):
                mine = q[b:b + 1, 2 * h:2 * h + 2].float().numpy()
                k, v = want.values("k", b, h), want.values("v", b, h)
                o, _, p = ref.attention(mine, k, v, dim ** -0.5)
                size, _, _ = ref.attention(mine, k, np.abs(v), dim ** -0.5)
                # bf16's half unit, probabilities of 11 bits, scores good to 2^-18
                tol = 2.0 ** -8 * 1.01 * np.abs(o) + 2.0 ** -10 * size + 1e-7
                assert (np.abs(out[b, 2 * h:2 * h + 2] - o[0]) <= tol[0]).all()
                w = 0.9 * np.concatenate([weights[b][h], [0.0]]) + p
                # each step adds an error of a score's 2^-18 and of two roundings
                assert np.abs(got[b, h, :w.size] - w).max() <= 2.0 ** -17 * (step + 1)
                # the reference goes on from the device's weights: choices are compared exactly
                weights[b][h] = got[b, h, :w.size].astype(np.float64)
        if step % 5 == 4:
            free = cache.pages_free
            held = [[got[b, h, :want.lens[b]] for h in range(heads)] for b in range(batch)]
            cache.evict(budget, recent)
            want, kept = want.evict(held, budget, recent)
            weights = [[held[b][h][kept[b][h]].astype(np.float64) for h in range(heads)]
                       for b in range(batch)]
            assert cache.lengths == want.lens == cache.cache.lens.tolist()
            assert cache.pages_free >= free
            now = cache.weights.cpu().numpy()
            for b in range(batch):
                for h in range(heads):
                    assert np.array_equal(now[b, h, :want.lens[b]], weights[b][h].astype(np.float32))
                    assert not now[b, h, want.lens[b]:].any()
        k, v = cache.read(torch.float32)
        for b in range(batch):
            for h in range(heads):
                n = want.lens[b]
                assert np.array_equal(k[b, :n, h].cpu().numpy(), want.values("k", b, h))
                assert np.array_equal(v[b, :n, h].cpu().numpy(), want.values("v", b, h))
    # what was read goes through the codec like any other rows
    k, _ = cache.read()
    rows = k.view(-1, heads * dim).view(torch.int16).cpu().numpy().view(np.uint16)
    again = CompressedTensor.from_words(rows, ibp.BF16, 0.9, 64, dev)
    back = again.empty_like(dev)
    again.decompress_into(back)
    assert np.array_equal(back.cpu().numpy().view(np.uint16), rows)
    cache.check()


def test_pool_limits():
    cache = DecodeCache(n_pages=4, batch=2, n_heads=1, head_dim=64, max_tokens=40, page_tokens=16)
    rows = torch.zeros((2 * 30, 1, 64), device="cuda")
    cache.append(rows, rows)
    assert cache.pages_free == 0 and cache.lengths == [30, 30]
    with pytest.raises(RuntimeError, match="pages are needed"):
        cache.evict(20, 2)
    with pytest.raises(RuntimeError, match="pages are needed"):
        cache.append(rows[:6], rows[:6])
    with pytest.raises(ValueError, match="would hold"):
        cache.append(rows[:40], rows[:40])
    with pytest.raises(ValueError, match="counts"):
        cache.append(rows[:5], rows[:5])
    cache.append(rows[:4], rows[:4], counts=[2, 2])
    assert cache.lengths == [32, 32]
    cache.check()
    plain = DecodeCache(n_pages=2, batch=1, n_heads=1, head_dim=64, max_tokens=16, page_tokens=16,
                        track_weights=False)
    with pytest.raises(RuntimeError, match="weights"):
        plain.evict(4, 1)
