"""Arguments of the 8-bit cache's calls that would have threads write over one another are
refused before a launch, and layouts that only look like it are not (needs a GPU: without one
every call is refused for its pointers)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lossless_bit_level_gb300 as ibp
from kv_harness import cache_of, pools, rounded
from test_gpu_kv import check_attention, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def case():
    rng = np.random.default_rng(0)
    want = cache_of(rng, [90, 33], 2, 16, 64, "int8")
    return want, pools(want, rng), rounded(rng.standard_normal((6, 4, 64)), "bf16").cuda()


@pytest.mark.parametrize("strides", [(0, 64), (64, 64), (256, 0), (256, 32), (0, 0), (128, 64),
                                     (192, 64), (64, 128), (192, 128)])
def test_outputs_over_one_another(case, strides):
    _, cache, q = case
    room = torch.zeros(6 * 1024, dtype=torch.bfloat16, device="cuda")
    out = room.as_strided((6, 4, 64), (*strides, 1))
    with pytest.raises(ibp.IBPError):
        run_attention(cache, q, [3, 3], 0.125, weights=False, out=out)
    assert not room.any()


@pytest.mark.parametrize("strides", [(256, 64), (64, 384), (512, 128), (128, 832), (192, 1216),
                                     (320, 128), (320, 256)])
def test_outputs_beside_one_another(case, strides):
    """Rows of heads, heads of rows, and the two interleaved."""
    want, cache, q = case
    room = torch.zeros(8 * 1024, dtype=torch.bfloat16, device="cuda")
    out = room.as_strided((6, 4, 64), (*strides, 1))
    got, lse, _, _ = run_attention(cache, q, [3, 3], 0.125, weights=False, out=out)
    check_attention(want, q, [3, 3], 0.125, got, lse, None, None)


def test_eviction_over_its_own_weights(case):
    _, cache, _ = case
    scratch = torch.empty(ibp.kv_evict_scratch_bytes(cache, 40), dtype=torch.uint8, device="cuda")
    n = 2 * 2 * cache.capacity
    room = torch.rand(2 * n, device="cuda")
    w = room[:n].view(2, 2, -1)
    dst = ibp.KVCache(*(torch.zeros_like(t) for t in (cache.k_codes, cache.v_codes, cache.k_scales,
                                                      cache.v_scales)),
                      cache.table.clone(), torch.zeros_like(cache.lens))
    for at in (0, 1, n - 1):
        new = room[at:at + n].view(2, 2, -1)
        with pytest.raises(ibp.IBPError):
            ibp.kv_evict(cache, w, 40, 8, dst, scratch, new_weights=new)
    ibp.kv_evict(cache, w, 40, 8, dst, scratch, new_weights=room[n:].view(2, 2, -1))
    assert dst.lens.tolist() == [40, 33]
