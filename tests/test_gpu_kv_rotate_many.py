"""Appending with a rotation where there are so many queries (over 16 MB) that they are rotated in a
launch of their own, which starts along with the one that appends (needs a GPU). Everything is
compared exactly, as in test_gpu_kv_rotate.py, from copies that are made right behind the call."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_rotate_reference as turn
import lossless_bit_level_gb300 as ibp
from kv_harness import DTYPES, cache_of, pools, random_rows, read_all, rounded, with_lens
from test_gpu_kv import status_word
from test_gpu_kv_select import bounds_of

pytestmark = pytest.mark.gpu

CASES = [
    # (lengths before, rows each, rows before and behind them, heads, query heads, page, dim, dtype, rotated,
    #  axes, interleaved, in place)
    ([30, 0, 100], [500, 77, 540], (3, 5), 2, 64, 64, 128, "bf16", 128, 1, False, False),
    ([30, 0, 100], [500, 0, 617], (0, 9), 2, 64, 32, 128, "fp16", 128, 3, False, True),
    ([7, 16], [200, 420], (1, 0), 4, 64, 16, 128, "fp32", 96, 2, True, False),
    ([3] * 300, [4, 5] * 150, (2, 2), 1, 66, 16, 128, "bf16", 64, 1, True, True),  # more offsets than are kept
    ([0], [2200], (0, 0), 2, 64, 128, 64, "fp16", 64, 4, False, True),
    ([50, 128], [1100, 1100], (0, 0), 3, 63, 128, 64, "bf16", 48, 2, False, False),
]


def build(case, seed):
    lens, counts, (before, behind), heads, q_heads, page, dim, dtype, part, axes, inter, in_place = case
    rng = np.random.default_rng(seed)
    n = before + sum(counts) + behind
    assert n * q_heads * dim * torch.empty((), dtype=DTYPES[dtype]).element_size() > 16 << 20
    assert n >= len(lens) * (page // 4)  # not a few rows a sequence
    want = cache_of(rng, lens, heads, page, dim, "int8", dtype)
    cache = pools(want, rng, room=max(counts) + page)
    axis = list(rng.integers(0, axes, part // 2)) if axes > 1 else [0] * (part // 2)
    axis[0] = axes - 1
    turns = turn.table(2500, part)
    cu = torch.tensor(before + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    return rng, n, want, cache, axis, turns, cu


def expected(case, want, axis, turns, place, k, v, q, out):
    """The plain cache with the rows appended, and the rotated queries over what was in their place."""
    lens, counts, (before, _), *_, inter, _ = case
    kt = turn.rotated(k.float().numpy(), turns, place, axis, inter)
    at = before
    for b, m in enumerate(counts):
        if m:
            want.append(b, {"k": kt[at:at + m], "v": v[at:at + m].float().numpy()})
        at += m
    y = out.clone()
    y[before:at] = torch.from_numpy(turn.rotated(q.float().numpy(), turns, place, axis, inter)).to(q.dtype)[before:at]
    return y


def same(want, cache, new_lens):
    got = read_all(with_lens(cache, new_lens), max(want.lens))
    for name in "kv":
        for b in range(want.batch):
            for h in range(want.heads):
                assert np.array_equal(got[name][b, :want.lens[b], h], want.values(name, b, h)), (name, b, h)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_many_queries(case, given):
    lens, counts, (before, behind), heads, q_heads, page, dim, dtype, part, axes, inter, in_place = case
    rng, n, want, cache, axis, turns, cu = build(case, sum(counts) + dim + given)
    place = np.concatenate([np.zeros(before, int)] + [np.arange(a, a + m) for a, m in zip(lens, counts)] +
                           [np.zeros(behind, int)])
    place = rng.integers(0, 2500, (n, axes)) if given else np.repeat(place[:, None], axes, 1)
    rows, q = random_rows(rng, n, heads, dim, dtype), rounded(rng.standard_normal((n, q_heads, dim)), dtype)
    start = torch.full_like(q, 5.0) if not in_place else q
    exp = expected(case, want, axis, turns, place, rows["k"], rows["v"], q, start)
    k, v, qd = rows["k"].cuda(), rows["v"].cuda(), q.cuda()
    out = qd if in_place else start.cuda()
    new_lens, status = torch.full_like(cache.lens, -7), status_word()
    rotation = ibp.KVRotation(torch.from_numpy(turns).cuda(), axis=axis, interleaved=inter)
    positions = torch.from_numpy(place.astype(np.int32)).cuda() if given else None
    heavy = torch.randn((4096, 4096), device="cuda")
    torch.mm(heavy, heavy, out=heavy.new_empty(heavy.shape))  # the stream is behind the host
    ibp.kv_append_rotated(cache, k, v, rotation, positions=positions, q=qd, q_out=None if in_place else out, cu=cu,
                          new_lens=new_lens, status=status)
    after, turned = new_lens.clone(), out.clone()
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and after.tolist() == want.lens
    assert torch.equal(turned.cpu(), exp)
    same(want, cache, after)


@pytest.mark.parametrize("case", [CASES[0], CASES[3]])
def test_many_queries_captured(case):
    """Captured once with what follows, replayed with other rows over the same cache."""
    lens, counts, (before, behind), heads, q_heads, page, dim, dtype, part, axes, inter, in_place = case
    rng, n, want, cache, axis, turns, cu = build(case, 1)
    place = np.concatenate([np.zeros(before, int)] + [np.arange(a, a + m) for a, m in zip(lens, counts)] +
                           [np.zeros(behind, int)])[:, None]
    k = torch.zeros((n, heads, dim), dtype=DTYPES[dtype], device="cuda")
    v, q = torch.zeros_like(k), torch.zeros((n, q_heads, dim), dtype=DTYPES[dtype], device="cuda")
    out = q if in_place else torch.full_like(q, 5.0)
    new_lens, after, turned = torch.empty_like(cache.lens), torch.empty_like(cache.lens), torch.empty_like(q)
    saved = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)]
    rotation = ibp.KVRotation(torch.from_numpy(turns).cuda(), axis=axis, interleaved=inter)

    def step():
        ibp.kv_append_rotated(cache, k, v, rotation, q=q, q_out=None if in_place else out, cu=cu, new_lens=new_lens)
        after.copy_(new_lens)
        turned.copy_(out)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for i in range(3):
        rows, fresh = random_rows(rng, n, heads, dim, dtype), rounded(rng.standard_normal((n, q_heads, dim)), dtype)
        for t, x in zip((cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales), saved):
            t.copy_(x)
        k.copy_(rows["k"]), v.copy_(rows["v"]), q.copy_(fresh)
        if not in_place:
            out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        again = build(case, 1)[2]  # the plain cache before the rows
        exp = expected(case, again, axis, turns, place, rows["k"], rows["v"], fresh,
                       fresh if in_place else torch.full_like(fresh, 5.0))
        assert torch.equal(turned.cpu(), exp) and after.tolist() == again.lens
        same(again, cache, after)


@pytest.mark.parametrize("in_place", [False, True])
def test_selection_right_behind_an_append_with_many_queries(in_place):
    """As in test_gpu_kv_operators_order.py, with so many queries that their launch comes between:
    scales that the append raises are read as they are after it."""
    batch, heads, q_heads, d, page, old, new = 24, 32, 96, 128, 32, 20, 40
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rows(n, times, h=heads):
        return (times * torch.randn((n, h, d), generator=gen, device="cuda")).to(torch.bfloat16)

    n_pages = 2 * batch
    codes = [torch.zeros((n_pages, heads, page, d), dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((n_pages, heads), device="cuda") for _ in range(2)]
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").view(batch, 2)
    lens = [torch.full((batch,), n, dtype=torch.int32, device="cuda") for n in (0, old, old + new)]
    caches = [ibp.KVCache(*codes, *scales, table, x) for x in lens]
    turn_ = ibp.KVRotation(ibp.rotation_table(old + new, d))
    ibp.kv_append(caches[0], rows(batch * old, 1.0), rows(batch * old, 1.0))
    start = [t.clone() for t in (*codes, *scales)]
    k, v, wide = rows(batch * new, 30.0), rows(batch * new, 30.0), rows(batch * new, 1.0, q_heads)
    assert wide.nbytes > 16 << 20
    place, q = torch.empty_like(wide), rows(batch, 1.0)
    out, bounds = torch.empty_like(q), bounds_of(caches[0])
    columns = torch.empty((batch, heads, 2), dtype=torch.int32, device="cuda")
    one = torch.zeros((batch, heads, 2), dtype=torch.int32, device="cuda") + torch.arange(2, device="cuda").int()
    scratch = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")

    def run(wait):
        for t, x in zip((*codes, *scales), start):
            t.copy_(x)
        place.copy_(wide) if in_place else place.fill_(3.0)
        ibp.kv_append_rotated(caches[1], k, v, turn_, q=place if in_place else wide,
                              q_out=None if in_place else place)
        if wait:
            torch.cuda.synchronize()
        ibp.kv_attention_selected(caches[2], one, q, out, 0.1, scratch)
        if wait:
            torch.cuda.synchronize()
        ibp.kv_bounds(caches[2], bounds)
        ibp.kv_select(caches[2], bounds, q, columns, scratch)
        return [t.clone() for t in (out, columns, bounds, place, *scales)]

    expected_ = run(True)
    assert (scales[0] > start[2]).any()
    heavy = torch.randn((4096, 4096), device="cuda")
    for i in range(20):
        torch.mm(heavy, heavy, out=heavy.new_empty(heavy.shape))
        for a, b in zip(run(False), expected_):
            assert torch.equal(a, b), i
