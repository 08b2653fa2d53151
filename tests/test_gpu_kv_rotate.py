"""Appending to the 8-bit key/value cache with the rotation of positions on the way, against
the plain rotation and the plain cache (needs a GPU). Every step is single precision as the
interface states it, so codes, scales and rotated queries are compared exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_rotate_reference as turn
import lossless_bit_level_gb300 as ibp
from kv_harness import DTYPES, cache_of, offsets, pools, random_rows, read_all, rounded, with_lens
from test_gpu_kv import status_word

pytestmark = pytest.mark.gpu


def numbers(counts, lens):
    """Token numbers of the rows [n, 1]."""
    return np.concatenate([np.arange(n, n + m) for n, m in zip(lens, counts)] or [np.zeros(0, int)])[:, None]


def run(want, cache, rows, q, counts, turns, axis=None, interleaved=False, positions=None, q_out=None,
        cu=True, times=1, code=0):
    """Appends, checks every page and the queries; positions [n, axes] or None."""
    lens = list(want.lens)
    rotation = ibp.KVRotation(torch.from_numpy(turns).cuda(), axis=axis, interleaved=interleaved)
    place = numbers(counts, lens) if positions is None else positions
    axis = axis or [0] * turns.shape[1]
    if positions is None:
        place = np.repeat(place, max(axis) + 1, 1)
    new_lens, status = torch.empty_like(cache.lens), status_word()
    k, v = rows["k"].cuda(), rows["v"].cuda()
    qd = None if q is None else q.cuda()
    out = None if q is None else torch.full_like(qd, 7.0) if q_out is None else q_out(qd)
    for _ in range(times):
        ibp.kv_append_rotated(
            cache, k, v, rotation, q=qd, q_out=out, cu=offsets(counts) if cu else None,
            positions=None if positions is None else torch.from_numpy(positions.astype(np.int32)).cuda(),
            new_lens=new_lens, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == code
    kt = turn.rotated(rows["k"].float().numpy(), turns, place, axis, interleaved)
    at = 0
    for b, n in enumerate(counts):
        if n:
            want.append(b, {"k": kt[at:at + n], "v": rows["v"][at:at + n].float().numpy()})
        at += n
    assert new_lens.tolist() == want.lens and cache.lens.tolist() == lens
    got = read_all(with_lens(cache, new_lens), max(want.lens) + 3)
    for name in "kv":
        for b in range(want.batch):
            for h in range(want.heads):
                n = want.lens[b]
                assert np.array_equal(got[name][b, :n, h], want.values(name, b, h)), (name, b, h)
                assert not got[name][b, n:, h].any()
    if q is not None:
        turned = turn.rotated(q.float().numpy(), turns, place, axis, interleaved)
        assert torch.equal(out.cpu(), torch.from_numpy(turned).to(q.dtype))


CASES = [
    # (lengths before, rows each, heads, query heads, page, dim, code, dtype, rotated, axes, interleaved)
    ([0], [1], 1, 1, 16, 64, "int8", "bf16", 64, 1, False),
    ([5, 0, 64, 63, 65], [1, 1, 1, 1, 1], 2, 8, 64, 128, "int8", "bf16", 128, 1, False),
    ([5, 0, 64, 63, 65], [130, 0, 1, 2, 63], 2, 6, 64, 128, "e4m3", "fp16", 128, 3, False),
    ([31, 33], [40, 7], 5, 5, 32, 64, "e4m3", "fp32", 32, 1, True),
    ([100, 7, 128], [29, 300, 0], 2, 14, 128, 128, "int8", "fp32", 48, 2, False),
    ([100, 7, 128], [29, 300, 0], 2, 2, 128, 128, "e4m3", "bf16", 128, 4, True),
    ([0, 0, 0], [70, 1, 16], 3, 9, 16, 128, "int8", "fp16", 16, 2, True),
    ([3, 15, 16], [17, 40, 33], 2, 4, 16, 64, "int8", "fp32", 64, 1, False),
    ([17, 300], [0, 0], 2, 2, 128, 64, "int8", "fp16", 64, 1, False),
    ([9, 2], [3, 2], 2, 32, 128, 128, "e4m3", "fp32", 112, 3, True),
]


@pytest.mark.parametrize("lens,counts,heads,q_heads,page,dim,code,dtype,part,axes,inter", CASES)
@pytest.mark.parametrize("given", [False, True])
def test_append_rotated_is_exact(lens, counts, heads, q_heads, page, dim, code, dtype, part, axes, inter, given):
    rng = np.random.default_rng(sum(lens) + sum(counts) + dim + part)
    want = cache_of(rng, lens, heads, page, dim, code, dtype)
    cache = pools(want, rng, room=max(counts) + page)
    rows, n = random_rows(rng, sum(counts), heads, dim, dtype), sum(counts)
    q = rounded(rng.standard_normal((n, q_heads, dim)), dtype)
    axis = list(rng.integers(0, axes, part // 2)) if axes > 1 else None
    if axis:
        axis[0] = axes - 1  # every axis is named
    positions = rng.integers(0, 700, (n, axes)) if given else None
    run(want, cache, rows, q, counts, turn.table(700, part), axis, inter, positions, times=2)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("axis", [[0] * 16 + [1] * 24 + [2] * 24, [i % 3 for i in range(64)]])
def test_axes_in_sections_and_in_turn(page, axis):
    """Units of eight pairs on one axis, and pairs on axes in turn."""
    rng = np.random.default_rng(page)
    lens, counts = [20, 0], [200, 77]
    want = cache_of(rng, lens, 2, page, 128, "int8")
    cache = pools(want, rng, room=max(counts) + page)
    rows = random_rows(rng, sum(counts), 2, 128)
    q = rounded(rng.standard_normal((sum(counts), 4, 128)), "bf16")
    run(want, cache, rows, q, counts, turn.table(300, 128), axis, False, rng.integers(0, 300, (277, 3)))


def test_far_positions():
    """A table over 2,000,001 positions: its angles are those of 64 bits."""
    rng = np.random.default_rng(1)
    want = cache_of(rng, [3], 2, 16, 64, "int8")
    cache = pools(want, rng, room=32)
    rows, q = random_rows(rng, 9, 2, 64), rounded(rng.standard_normal((9, 4, 64)), "bf16")
    table = ibp.rotation_table(2_000_001, 64)
    for p in (0, 1, 65_535, 65_536, 1_999_999, 2_000_000):
        angle = p * 10000.0 ** (-np.arange(32) / 32)
        # rounding, and the last bits of the two libraries' 64-bit powers times the position
        assert np.allclose(table[p].cpu().numpy(), np.stack([np.cos(angle), np.sin(angle)], 1),
                           rtol=0, atol=2.0 ** -24 + p * 2.0 ** -50)
    where = np.array([[0], [1], [1_999_999], [2_000_000], [65_535], [65_536], [7], [1_234_567], [3]])
    run(want, cache, rows, q, [9], table.cpu().numpy(), positions=where)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("each", [1, 37])
def test_same_count_each_views_and_another_stream(dtype, each):
    """No offsets; k, v and q views of one fused tensor, q rotated in place; a stream of its own."""
    rng = np.random.default_rng(each)
    lens, heads, page, dim = [3, 40, 0], 2, 32, 64
    want = cache_of(rng, lens, heads, page, dim, "int8")
    cache = pools(want, rng, room=64)
    fused = rounded(rng.standard_normal((3 * each, 10, dim)), dtype)
    turns = turn.table(100, 64)
    dev, table = fused.cuda(), torch.from_numpy(turns).cuda()
    new_lens, status = torch.empty_like(cache.lens), status_word()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    ibp.kv_append_rotated(cache, dev[:, 1:5:2], dev[:, 8:10], ibp.KVRotation(table), q=dev[:, 5:8],
                          new_lens=new_lens, status=status, stream=stream)
    stream.synchronize()
    assert int(status.item()) == 0
    place = numbers([each] * 3, lens)
    k = turn.rotated(fused[:, 1:5:2].float().numpy(), turns, place, [0] * 32, False)
    for b in range(3):
        at = slice(b * each, (b + 1) * each)
        want.append(b, {"k": k[at], "v": fused[at, 8:10].float().numpy()})
    got = read_all(with_lens(cache, new_lens), max(want.lens))
    for name in "kv":
        for b in range(3):
            for h in range(heads):
                assert np.array_equal(got[name][b, :want.lens[b], h], want.values(name, b, h))
    q = turn.rotated(fused[:, 5:8].float().numpy(), turns, place, [0] * 32, False)
    assert torch.equal(dev[:, 5:8].cpu(), torch.from_numpy(q).to(DTYPES[dtype]))
    rest = [0, 1, 2, 3, 4, 8, 9]
    assert torch.equal(dev[:, rest].cpu(), fused[:, rest])


@pytest.mark.parametrize("few", [True, False])
def test_values_that_are_not_finite(few):
    """NaN and infinities go through the rotation, then follow the quantisation's rule."""
    rng = np.random.default_rng(8)
    lens, counts = [3, 0], ([2, 3] if few else [60, 33])
    want = cache_of(rng, lens, 2, 32, 64, "int8")
    cache = pools(want, rng, room=96)
    rows = random_rows(rng, sum(counts), 2, 64, "fp32")
    rows["k"][0, 0, 3], rows["k"][1, 1, 40], rows["k"][2, 0, 5] = np.inf, -np.inf, np.nan
    rows["k"][4, 1, 63] = 3e38
    rows["v"][1, 0, 0], rows["v"][3, 1, 9] = np.nan, np.inf
    run(want, cache, rows, None, counts, turn.table(100, 64))


def test_positions_outside_the_table_are_held_and_reported():
    rng = np.random.default_rng(2)
    want = cache_of(rng, [4], 1, 16, 64, "int8")
    cache = pools(want, rng, room=32)
    rows, q = random_rows(rng, 3, 1, 64), rounded(rng.standard_normal((3, 2, 64)), "bf16")
    run(want, cache, rows, q, [3], turn.table(50, 64), positions=np.array([[-1], [50], [7]]), code=ibp.ERR_INDEX)


def test_rows_of_no_sequence_and_rows_without_room():
    """Queries of rows before the first offset and behind the last stay; those whose token had
    no room are rotated all the same."""
    rng = np.random.default_rng(3)
    want = cache_of(rng, [10, 30], 2, 16, 64, "int8")
    cache = pools(want, rng, cols=2, room=1)
    turns = turn.table(100, 64)
    q = rounded(rng.standard_normal((11, 4, 64)), "bf16").cuda()
    rows = {n: t.cuda() for n, t in random_rows(rng, 11, 2, 64).items()}
    out, status = torch.full_like(q, 5.0), status_word()
    new_lens = torch.empty_like(cache.lens)
    cu = torch.tensor([2, 4, 9], dtype=torch.int32, device="cuda")
    ibp.kv_append_rotated(cache, rows["k"], rows["v"], ibp.KVRotation(torch.from_numpy(turns).cuda()),
                          q=q, q_out=out, cu=cu, new_lens=new_lens, status=status)
    assert int(status.item()) == ibp.ERR_INDEX and new_lens.tolist() == [12, 32]
    place = np.array([0, 0, 10, 11, 30, 31, 32, 33, 34, 0, 0])[:, None]
    turned = torch.from_numpy(turn.rotated(q.float().cpu().numpy(), turns, place, [0] * 32, False)).bfloat16()
    assert torch.equal(out[2:9].cpu(), turned[2:9])
    assert bool((out[:2] == 5).all()) and bool((out[9:] == 5).all())


def test_table_refusals_on_the_gpu():
    """What looks like q beside q_out and is not."""
    rng = np.random.default_rng(4)
    cache = pools(cache_of(rng, [4], 1, 16, 64, "int8"), rng, room=32)
    rows = {n: t.cuda() for n, t in random_rows(rng, 2, 1, 64).items()}
    rotation = ibp.KVRotation(ibp.rotation_table(64, 64))
    room = torch.zeros(1024, dtype=torch.bfloat16, device="cuda")
    q = room[:256].view(2, 2, 64)
    for out in (room[8:264].view(2, 2, 64), room[128:384].view(2, 2, 64),
                room.as_strided((2, 2, 64), (64, 64, 1))):
        with pytest.raises(ibp.IBPError):
            ibp.kv_append_rotated(cache, rows["k"], rows["v"], rotation, q=q, q_out=out)
    ibp.kv_append_rotated(cache, rows["k"], rows["v"], rotation, q=q, q_out=room[256:512].view(2, 2, 64))


def test_in_a_graph():
    """Captured once, replayed with other rows."""
    rng = np.random.default_rng(5)
    lens, counts = [30, 2], [1, 1]
    first = cache_of(rng, lens, 2, 32, 128, "e4m3")
    cache = pools(first, rng, room=32)
    k = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    v, q = torch.zeros_like(k), torch.zeros((2, 6, 128), dtype=torch.bfloat16, device="cuda")
    out, new_lens, status = torch.zeros_like(q), torch.empty_like(cache.lens), status_word()
    turns = turn.table(64, 128)
    rotation, cu = ibp.KVRotation(torch.from_numpy(turns).cuda()), offsets(counts)
    call = lambda: ibp.kv_append_rotated(cache, k, v, rotation, q=q, q_out=out, cu=cu,  # noqa: E731
                                         new_lens=new_lens, status=status)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    rows, new_q = random_rows(rng, 2, 2, 128), rounded(rng.standard_normal((2, 6, 128)), "bf16")
    k.copy_(rows["k"]), v.copy_(rows["v"]), q.copy_(new_q)
    graph.replay()
    torch.cuda.synchronize()
    place = numbers(counts, lens)
    kt = turn.rotated(rows["k"].float().numpy(), turns, place, [0] * 64, False)
    for b in range(2):
        first.append(b, {"k": kt[b:b + 1], "v": rows["v"][b:b + 1].float().numpy()})
    got = read_all(with_lens(cache, new_lens), 31)
    for b in range(2):
        for h in range(2):
            assert np.array_equal(got["k"][b, :first.lens[b], h], first.values("k", b, h))
    assert torch.equal(out.cpu(), torch.from_numpy(
        turn.rotated(new_q.float().numpy(), turns, place, [0] * 64, False)).bfloat16())
