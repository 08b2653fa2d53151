"""What follows the 8-bit key/value cache's calls in a graph sees all that they wrote
(needs a GPU).

The second kernel of a call starts while the first one ends, and a graph's next node is
ordered behind the second alone: it has to wait for the first in every block, also in calls
that leave it nothing to do (every segment finished by one CTA; nothing kept). So the next
node of each graph here copies what the call wrote, and the copies are looked at."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
import lossless_bit_level_gb300 as ibp
from kv_harness import cache_of, pools, rounded, with_lens
from test_gpu_kv import check_attention, status_word

pytestmark = pytest.mark.gpu


def captured(call):
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("batch,longest,n", [(1, 64, 1), (40, 64, 2), (5, 700, 3), (2, 130, 70)])
def test_attention_copied_by_the_next_node(batch, longest, n, weights):
    rng = np.random.default_rng(batch + longest)
    heads, q_heads, dim = 2, 4, 64
    lens = [longest] + [int(x) for x in rng.integers(0, longest + 1, batch - 1)]
    want = cache_of(rng, lens, heads, 16, dim, "int8")
    cache = pools(want, rng)
    q = rounded(rng.standard_normal((batch * n, q_heads, dim)), "bf16").cuda()
    out, lse, status = torch.empty_like(q), torch.empty((batch * n, q_heads), device="cuda"), status_word()
    w = torch.zeros((batch, heads, cache.capacity), device="cuda") if weights else None
    w_in = None if w is None else torch.rand_like(w)
    copies = [torch.empty_like(t) for t in (out, lse) + ((w,) if weights else ())]
    scratch = torch.empty(ibp.kv_attention_scratch_bytes(cache, batch * n, n, q_heads, weights),
                          dtype=torch.uint8, device="cuda")

    def call():
        for t in (out, lse) + ((w,) if weights else ()):
            t.fill_(-3.0)
        ibp.kv_attention(cache, q, out, 0.125, scratch, max_q=n, lse=lse, weights=w,
                         weights_in=w_in, decay=0.5, status=status)
        for to, t in zip(copies, (out, lse, w)):
            to.copy_(t)

    graph = captured(call)
    for _ in range(5):
        for t in copies:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        check_attention(want, q, [n] * batch, 0.125, copies[0], copies[1],
                        copies[2] if weights else None, w_in)
    assert int(status.item()) == 0


@pytest.mark.parametrize("lens", [[0, 0, 0], [0, 5, 90]])
def test_eviction_copied_by_the_next_node(lens):
    rng = np.random.default_rng(sum(lens))
    heads, page, dim, budget = 3, 16, 64, 40
    src = cache_of(rng, [90] * 3, heads, page, dim, "int8")
    cache = pools(src, rng)
    cache = with_lens(cache, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    dst = pools(ref.Cache(3, heads, page, dim, "int8"), rng, room=budget)
    weights = torch.rand((3, heads, cache.capacity), device="cuda")
    new_w = torch.empty((3, heads, budget), device="cuda")
    kept = torch.empty((3, heads, budget), dtype=torch.int32, device="cuda")
    scratch = torch.empty(ibp.kv_evict_scratch_bytes(cache, budget), dtype=torch.uint8, device="cuda")
    status, copies = status_word(), [torch.empty_like(t) for t in (dst.lens, new_w, kept)]

    def call():
        dst.lens.fill_(-9)
        new_w.fill_(-9.0)
        kept.fill_(-9)
        ibp.kv_evict(cache, weights, budget, 8, dst, scratch, new_weights=new_w, kept=kept, status=status)
        for to, t in zip(copies, (dst.lens, new_w, kept)):
            to.copy_(t)

    graph = captured(call)
    for _ in range(5):
        for t in copies:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got_lens, got_w, got_kept = (t.cpu() for t in copies)
        assert got_lens.tolist() == [min(n, budget) for n in lens]
        for b, n in enumerate(lens):
            m = min(n, budget)
            assert (got_kept[b, :, m:] == -1).all() and (got_w[b, :, m:] == 0).all()
            at = got_kept[b, :, :m].long()
            assert (at >= 0).all() and torch.equal(got_w[b, :, :m], weights[b].cpu().gather(1, at))
    assert int(status.item()) == 0
