"""Where rotated queries may be written (needs a GPU): never over rows that are still read, and
anywhere beside them, in one fused tensor too. Results are compared exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_rotate_reference as turn
import lossless_bit_level_gb300 as ibp
from kv_harness import cache_of, pools, rounded

pytestmark = pytest.mark.gpu

DIM = 64


def setup(n):
    rng = np.random.default_rng(n)
    cache = pools(cache_of(rng, [4], 2, 16, DIM, "int8"), rng, room=n + 16)
    turns = turn.table(64, DIM)
    return rng, cache, turns, ibp.KVRotation(torch.from_numpy(turns).cuda())


@pytest.mark.parametrize("n", [1, 2, 30])
def test_over_keys_or_values(n):
    rng, cache, _, rotation = setup(n)
    fused = rounded(rng.standard_normal((n, 12, DIM)), "bf16").cuda()
    before, scales = fused.clone(), cache.k_scales.clone()
    part = lambda a, b, step=1: fused[:, a:b:step]  # noqa: E731
    apart = rounded(rng.standard_normal((n, 2, DIM)), "bf16").cuda()
    flat = fused.view(-1)
    for q, out, k, v in (
            (part(0, 2), None, part(0, 2), part(4, 6)),             # the keys themselves
            (part(0, 2), None, part(4, 6), part(1, 3)),             # values over the last of q's heads
            (apart, part(0, 2), part(1, 3), part(4, 6)),
            (apart, part(3, 7, 3), part(0, 2), part(5, 8, 1)[:, 1:]),  # heads 3 and 6; 6 and 7
            (apart, flat[8:8 + 2 * DIM].expand(n, -1).view(n, 2, DIM) if n == 1 else part(4, 6), part(0, 2), part(5, 7)),
            (apart, part(0, 4, 3), part(3, 5), part(6, 8)),
            (apart, part(0, 2), fused[:1, 1:3].expand(n, 2, DIM), part(4, 6)),  # one row of K for all
            (apart, part(0, 2), part(4, 6), fused[:, 1:2].expand(n, 2, DIM)),   # one head of V for all
    ):
        with pytest.raises(ibp.IBPError):
            ibp.kv_append_rotated(cache, k, v, rotation, q=q, q_out=out)
    if n > 1:  # rows of another stride among the keys'
        with pytest.raises(ibp.IBPError):
            ibp.kv_append_rotated(cache, part(0, 2), part(4, 6), rotation, q=apart,
                                  q_out=flat[2 * DIM:].as_strided((n, 2, DIM), (2 * DIM, DIM, 1)))
    torch.cuda.synchronize()
    assert torch.equal(fused, before)  # nothing was launched
    assert torch.equal(cache.k_scales.nan_to_num(-1), scales.nan_to_num(-1))


@pytest.mark.parametrize("n", [1, 2, 30])
def test_beside_keys_and_values(n):
    rng, cache, turns, rotation = setup(n)
    place = 4 + np.arange(n)[:, None]
    for q_heads, k_heads, v_heads, out_heads in (
            ([4, 5, 6], [0, 1], [2, 3], None),                      # in place, behind them
            ([1, 4, 7], [0, 3], [2, 5], None),                      # every third, each
            ([0, 1, 2], [6, 7], [8, 9], [3, 4, 5]),                 # q, then its place, then K and V
            ([9, 10, 11], [2, 4], [1, 3], [6, 7, 8]),
            ([9, 10, 11], [1, 5], [4, 8], [0, 3, 6]),               # K's heads between those of out
            ([0, 1], [4, 4], [2, 2], [10, 11]),                     # one head for all
    ):
        fused = rounded(rng.standard_normal((n, 12, DIM)), "bf16")
        dev = fused.cuda()

        def part(heads):
            step = heads[1] - heads[0]
            return dev[:, heads[0]:heads[0] + 1].expand(n, len(heads), DIM) if step == 0 else \
                dev[:, heads[0]:heads[-1] + 1:step]

        ibp.kv_append_rotated(cache, part(k_heads), part(v_heads), rotation, q=part(q_heads),
                              q_out=None if out_heads is None else part(out_heads))
        want = fused.clone()
        want[:, out_heads or q_heads] = torch.from_numpy(
            turn.rotated(fused[:, q_heads].float().numpy(), turns, place, [0] * (DIM // 2), False)).bfloat16()
        assert torch.equal(dev.cpu(), want)
    # the same row of K for all, in the tensor whose first rows hold the queries
    dev = rounded(rng.standard_normal((n + 1, 2, DIM)), "bf16").cuda()
    ibp.kv_append_rotated(cache, dev[n:].expand(n, 2, DIM), dev[n:].expand(n, 2, DIM), rotation, q=dev[:n])
    torch.cuda.synchronize()
