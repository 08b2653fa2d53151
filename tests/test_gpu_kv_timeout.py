"""The bounded waits of the attention kernels run out on the GPU, and the stream and the
library stay usable afterwards (needs a GPU).

The testing hooks (include/ibp_testing.h) make the fetching warps stop after a CTA's first
tile -- the next barrier is one that nothing completes -- and lower the limit to 1 ms: the
waits run out, the call records IBP_ERR_TIMEOUT, every warp gives up and returns, and what
is in flight is waited for first. The next call on the same stream gives the same bits as
one before. No GPU fault, trap or endless wait is involved."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lossless_bit_level_gb300 as ibp
from kv_harness import TORCH_CODE, rounded
from test_gpu_kv import status_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,weights,dim", [(1, False, 128), (3, True, 64), (12, True, 128),
                                           (64, False, 128), (300, False, 64)])
def test_wait_runs_out_then_the_stream_recovers(n, weights, dim):
    rng = np.random.default_rng(n)
    batch, heads, q_heads, page = 4, 8, 8, 64
    lens = [20_000, 9_000, 33, 15_001]
    pages = [-(-t // page) for t in lens]
    g = torch.Generator(device="cuda").manual_seed(n)
    shape = (sum(pages), heads, page, dim)
    k, v = (torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8).view(
        TORCH_CODE["int8"]) for _ in range(2))
    ks, vs = (torch.rand(shape[:2], generator=g, device="cuda") * 0.01 for _ in range(2))
    table = torch.full((batch, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = torch.arange(at, at + m)
        at += m
    cache = ibp.KVCache(k, v, ks, vs, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    q = rounded(rng.standard_normal((batch * n, q_heads, dim)), "bf16").cuda()
    scratch = torch.zeros(ibp.kv_attention_scratch_bytes(cache, batch * n, n, q_heads, weights),
                          dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def call():
        status, out = status_word(), torch.zeros_like(q)
        w = torch.zeros((batch, heads, cache.capacity), device="cuda") if weights else None
        stream.wait_stream(torch.cuda.current_stream())
        ibp.kv_attention(cache, q, out, 0.1, scratch, max_q=n, weights=w, status=status, stream=stream)
        stream.synchronize()  # the call ends: no wait is left without a bound
        return int(status.item()), out, w

    before = call()
    assert before[0] == 0 and torch.isfinite(before[1].float()).all()
    limit, held = ibp.testing_set_wait_limit_ns(1_000_000), ibp.testing_withhold_plans(True)
    try:
        assert call()[0] == ibp.ERR_TIMEOUT
    finally:
        ibp.testing_withhold_plans(held)
        ibp.testing_set_wait_limit_ns(limit)
    after = call()
    assert after[0] == 0 and torch.equal(before[1], after[1])
    if weights:
        assert torch.equal(before[2], after[2])
