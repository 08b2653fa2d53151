"""Attention of batches that share beginnings over the 8-bit key/value cache, against plain
attention of each sequence in 64 bits (needs a GPU). Tolerances are those of test_gpu_kv.py with
one more rounding of 2^-22 of the output: a row's two halves are joined in single precision."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
import lossless_bit_level_gb300 as ibp
from kv_harness import as_float32, offsets, pools, random_rows, rounded, with_lens
from test_gpu_kv import check_attention, run_attention, status_word

pytestmark = pytest.mark.gpu


def shared_cache(rng, groups, heads, page, dim, code, spare=2, wide=True):
    """groups: [(prefix, [own tokens of each sequence])]; the plain cache and the same as pools in
    which a group's whole prefix pages are there once (what would be the others' is NaN scales).
    wide: tables of so many columns (most of them unused) that the call is divided."""
    lens = [p + t for p, own in groups for t in own]
    want = ref.Cache(len(lens), heads, page, dim, code)
    b = 0
    for p, own in groups:
        prefix = as_float32(random_rows(rng, p, heads, dim))
        for t in own:
            if p:
                want.append(b, prefix)
            if t:
                want.append(b, as_float32(random_rows(rng, t, heads, dim)))
            b += 1
    cols = (64 << 20) // (len(lens) * page * heads * 2 * dim) + 1 if wide else None
    cache = pools(want, rng, spare=spare, cols=cols)
    b = 0
    for p, own in groups:
        for i in range(1, len(own)):
            n = p // page
            old = cache.table[b + i, :n].long()
            cache.k_scales[old] = float("nan")
            cache.v_scales[old] = float("nan")
            cache.table[b + i, :n] = cache.table[b, :n]
        b += len(own)
    return want, cache


def run_shared(cache, groups, q, counts, scale, prefix=None, offsets_of=None, cu=True, group_rows=None, out=None,
               status=None, stream=None):
    sizes = [len(own) for _, own in groups]
    starts = np.concatenate([[0], np.cumsum(sizes)]) if offsets_of is None else np.array(offsets_of)
    prefix = [p for p, _ in groups] if prefix is None else prefix
    if group_rows is None:
        group_rows = max((sum(counts[a:b]) for a, b in zip(starts[:-1], starts[1:])), default=0)
    n, heads, max_q = q.shape[0], q.shape[1], max(counts, default=0)
    size = ibp.kv_attention_shared_scratch_bytes(cache, n, max_q, heads, len(prefix), group_rows)
    scratch = torch.empty(max(16, size), dtype=torch.uint8, device="cuda").fill_(0xFF)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((n, heads), 7.0, device="cuda")
    own = status_word() if status is None else status
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    ibp.kv_attention_shared(cache, q, out, scale, scratch,
                            torch.tensor(starts, dtype=torch.int32, device="cuda"),
                            torch.tensor(prefix, dtype=torch.int32, device="cuda"), group_rows,
                            cu_q=offsets(counts) if cu else None, max_q=max_q, lse=lse, status=own, stream=stream)
    torch.cuda.synchronize()
    if status is None:
        assert int(own.item()) == 0
    return out, lse


CASES = [
    # (groups, query rows each, q heads, kv heads, dim, page, code, dtype)
    ([(64, [1, 2])], [1, 1], 1, 1, 128, 16, "int8", "bf16"),
    ([(777, [100, 1, 33, 16])], [1] * 4, 8, 2, 128, 16, "int8", "bf16"),
    ([(300, [7, 0, 50]), (0, [40, 3]), (130, [9])], [1] * 6, 4, 4, 64, 32, "e4m3", "fp16"),
    ([(1000, [0, 0, 0, 64, 5])], [1] * 5, 8, 1, 64, 64, "int8", "bf16"),         # 40 rows: the kernel for many
    ([(1500, [3, 200, 128, 10] * 5), (90, [30] * 3)], [1] * 23, 32, 2, 128, 64, "int8", "bf16"),
    ([(1111, [20, 9, 70] * 4), (640, [0, 1, 100] * 3)], [1] * 21, 16, 2, 128, 32, "e4m3", "bf16"),
    ([(513, [9, 40, 12, 70])], [3, 7, 1, 5], 8, 2, 64, 16, "int8", "fp16"),
    ([(513, [9, 2, 0, 70])], [3, 7, 1, 5], 16, 1, 64, 128, "e4m3", "fp16"),       # rows within the prefix
    ([(400, [100, 33, 90])], [16, 9, 12], 16, 4, 128, 64, "int8", "bf16"),        # 64 rows a sequence
    ([(200, [100, 90])], [90, 33], 8, 4, 128, 64, "int8", "bf16"),                # more: undivided
    ([(40, [5, 0, 1])], [4, 0, 2], 4, 2, 64, 16, "int8", "bf16"),                 # one without rows
    ([(20, [5, 1]), (0, [0, 0])], [30, 2, 3, 1], 2, 2, 64, 16, "int8", "fp16"),   # rows that see nothing
    ([(2000, [60] * 70)], [1] * 70, 4, 1, 64, 64, "int8", "fp16"),                # 280 rows: two blocks
]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("groups,counts,q_heads,heads,dim,page,code,dtype", CASES)
def test_shared_beginnings(groups, counts, q_heads, heads, dim, page, code, dtype, wide):
    rng = np.random.default_rng(sum(counts) + dim + page + q_heads)
    want, cache = shared_cache(rng, groups, heads, page, dim, code, wide=wide)
    q = rounded(1.5 * rng.standard_normal((sum(counts), q_heads, dim)), dtype).cuda()
    out, lse = run_shared(cache, groups, q, counts, dim ** -0.5)
    check_attention(want, q, counts, dim ** -0.5, out, lse, None, None)
    again, _ = run_shared(cache, groups, q, counts, dim ** -0.5)
    assert torch.equal(out, again)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 4.0])
@pytest.mark.parametrize("many", [False, True])
def test_other_scales(scale, many):
    rng = np.random.default_rng(1)
    groups = [(320, [11, 40, 3] * (4 if many else 1))]
    n = len(groups[0][1])
    want, cache = shared_cache(rng, groups, 2, 32, 128, "int8")
    q = rounded(0.5 * rng.standard_normal((n, 8, 128)), "bf16").cuda()
    out, lse = run_shared(cache, groups, q, [1] * n, scale)
    # a negative scale is the positive one on rows of the other sign
    check_attention(want, q if scale >= 0 else -q, [1] * n, abs(scale), out, lse, None, None)


def test_wrong_bounds_and_prefixes_choose_another_way_only():
    """group_rows too small or too large, and prefixes longer than what the rows see."""
    rng = np.random.default_rng(2)
    groups, counts = [(500, [9, 1, 30] * 5)], [2, 1, 3] * 5
    want, cache = shared_cache(rng, groups, 2, 16, 64, "int8")
    q = rounded(rng.standard_normal((sum(counts), 8, 64)), "bf16").cuda()
    for group_rows in (0, 1, 7, 30, 1 << 30):
        out, lse = run_shared(cache, groups, q, counts, 0.125, group_rows=group_rows)
        check_attention(want, q, counts, 0.125, out, lse, None, None)
    for prefix in (0, 15, 16, 496, -3):
        out, lse = run_shared(cache, groups, q, counts, 0.125, prefix=[prefix])
        check_attention(want, q, counts, 0.125, out, lse, None, None)
    # equal sequences: everything is shared, a prefix past the length counts as far as rows see it
    groups = [(160, [0, 0, 0])]
    want, cache = shared_cache(rng, groups, 2, 16, 64, "int8")
    for counts in ([1, 1, 1], [17, 1, 33]):
        q = rounded(rng.standard_normal((sum(counts), 4, 64)), "bf16").cuda()
        out, lse = run_shared(cache, groups, q, counts, 0.125, prefix=[100_000])
        check_attention(want, q, counts, 0.125, out, lse, None, None)


def test_sequences_of_no_group_and_other_rows():
    """Groups in the middle of the batch; rows before the first offset and behind the last stay."""
    rng = np.random.default_rng(3)
    groups = [(0, [70, 5]), (200, [9, 33, 1]), (0, [20])]
    want, cache = shared_cache(rng, groups, 2, 16, 64, "e4m3")
    q = rounded(rng.standard_normal((11, 4, 64)), "fp16").cuda()
    scratch = torch.empty(ibp.kv_attention_shared_scratch_bytes(cache, 11, 2, 4, 1, 4), dtype=torch.uint8,
                          device="cuda")
    cu = torch.tensor([2, 3, 4, 6, 7, 8, 9], dtype=torch.int32, device="cuda")
    out, lse, status = torch.full_like(q, 3.0), torch.full((11, 4), 3.0, device="cuda"), status_word()
    ibp.kv_attention_shared(cache, q, out, 0.2, scratch, torch.tensor([2, 5], dtype=torch.int32, device="cuda"),
                            torch.tensor([200], dtype=torch.int32, device="cuda"), 4, cu_q=cu, max_q=2, lse=lse,
                            status=status)
    assert int(status.item()) == 0
    check_attention(want, q[2:9], [1, 1, 2, 1, 1, 1], 0.2, out[2:9], lse[2:9], None, None)
    for t in (out, lse):
        assert bool((t[:2] == 3).all()) and bool((t[9:] == 3).all())


def test_more_sequences_than_one_slab():
    """300 sequences: groups cut by the slabs of 128, and one without any group between them."""
    rng = np.random.default_rng(4)
    groups = [(90, [3] * 120), (70, [1, 20] * 70), (0, [10]), (50, [2] * 39)]
    n = sum(len(own) for _, own in groups)
    want, cache = shared_cache(rng, groups, 1, 16, 64, "int8")
    q = rounded(rng.standard_normal((n, 2, 64)), "bf16").cuda()
    out, lse = run_shared(cache, groups, q, [1] * n, 0.125)
    check_attention(want, q, [1] * n, 0.125, out, lse, None, None)


@pytest.mark.parametrize("many", [False, True])
def test_views_no_offsets_and_another_stream(many):
    rng = np.random.default_rng(5)
    groups = [(256, [30, 60, 2] * (5 if many else 1))]
    n = len(groups[0][1])
    want, cache = shared_cache(rng, groups, 2, 64, 128, "int8")
    wide = rounded(rng.standard_normal((2 * n, 9, 128)), "bf16").cuda()
    room = torch.zeros((2 * n, 6, 128), dtype=torch.bfloat16, device="cuda")
    q, out = wide[:, 1:9:2], room[:, 1:5]
    _, lse = run_shared(cache, groups, q, [2] * n, 0.09, cu=False, out=out, stream=torch.cuda.Stream())
    check_attention(want, q, [2] * n, 0.09, out, lse, None, None)
    assert not room[:, 0].any() and not room[:, 5].any()


def test_bad_groups_pages_and_lengths_are_reported():
    rng = np.random.default_rng(6)
    groups, counts = [(200, [9, 33, 1, 40])], [1] * 4
    want, cache = shared_cache(rng, groups, 2, 16, 64, "int8")
    q = rounded(rng.standard_normal((4, 4, 64)), "fp16").cuda()

    def run(c, **kw):
        status = status_word()
        out, lse = run_shared(c, groups, q, counts, 0.125, status=status, **kw)
        return int(status.item()), out, lse

    for bad in ([0, 5], [-1, 4], [3, 1]):
        code, out, lse = run(cache, offsets_of=bad, prefix=[200], group_rows=4)
        assert code == ibp.ERR_INDEX and bool(torch.isfinite(out.float()).all())
    for prefix in ([100, 60], [0, 200]):  # not rising: the rows of a valid part are right all the same
        code, out, lse = run(cache, offsets_of=[0, 4, 2], prefix=prefix, group_rows=4)
        assert code == ibp.ERR_INDEX
    saved = cache.table.clone()
    cache.table[0, 2] = cache.k_codes.shape[0]
    code, out, _ = run(cache)
    assert code == ibp.ERR_INDEX and bool(torch.isfinite(out.float()).all())
    cache.table.copy_(saved)
    code, _, _ = run(with_lens(cache, torch.tensor([209, 100_000, 201, 240], dtype=torch.int32, device="cuda")))
    assert code == ibp.ERR_INDEX
    code, out, lse = run(cache)
    assert code == 0
    check_attention(want, q, counts, 0.125, out, lse, None, None)


@pytest.mark.parametrize("many", [False, True])
def test_captured_and_replayed_in_turn(many):
    """Two captured calls on one workspace, replayed in turn with other rows and longer sequences."""
    rng = np.random.default_rng(7)
    stream, steps = torch.cuda.Stream(), []
    scratch = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    for code in ("int8", "e4m3"):
        groups = [(330, [40, 7, 90] * (6 if many else 1)), (64, [1, 5])]
        n = sum(len(own) for _, own in groups)
        want, cache = shared_cache(rng, groups, 2, 16, 64, code)
        q = torch.zeros((n, 8, 64), dtype=torch.bfloat16, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((n, 8), device="cuda")
        starts = torch.tensor([0, n - 2, n], dtype=torch.int32, device="cuda")
        prefix = torch.tensor([330, 64], dtype=torch.int32, device="cuda")

        def step(cache=cache, q=q, out=out, lse=lse, starts=starts, prefix=prefix, n=n):
            ibp.kv_attention_shared(cache, q, out, 0.125, scratch, starts, prefix, n - 2, lse=lse)

        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        steps.append((graph, want, q, out, lse, n, step))
    for _ in range(3):
        for graph, _, q, _, _, n, _ in steps:
            q.copy_(rounded(rng.standard_normal((n, 8, 64)), "bf16"))
            graph.replay()
        torch.cuda.synchronize()
        for _, want, q, out, lse, n, _ in steps:
            check_attention(want, q, [1] * n, 0.125, out, lse, None, None)


def test_the_same_as_undivided():
    """No group at all: the plain call's results up to roundings."""
    rng = np.random.default_rng(8)
    groups = [(0, [500, 33, 0, 70])]
    want, cache = shared_cache(rng, groups, 2, 32, 64, "int8")
    q = rounded(rng.standard_normal((4, 4, 64)), "bf16").cuda()
    out, lse = run_shared(cache, [], q, [1] * 4, 0.125, group_rows=0)
    check_attention(want, q, [1] * 4, 0.125, out, lse, None, None)
    plain, plain_lse, _, _ = run_attention(cache, q, [1] * 4, 0.125, weights=False)
    half = 2.0 ** -8  # two roundings to bf16 of values 2^-20 apart
    assert bool(((out.float() - plain.float()).abs() <= 2.1 * half * plain.float().abs() + 2.0 ** -20).all())


@pytest.mark.parametrize("fill", [-1, 0])
@pytest.mark.parametrize("times", [1, 5])  # 10 and 50 rows a head
def test_a_group_whose_first_sequence_is_empty(times, fill):
    """A slot without rows or tokens at the head of a group: what its table holds is never read."""
    rng = np.random.default_rng(times)
    groups = [(320, [0] + [11, 40, 3, 70, 0] * times), (0, [5]), (200, [0, 9, 30])]
    counts = [0] + [1] * (5 * times) + [2] + [0, 1, 3]
    want, cache = shared_cache(rng, groups, 2, 32, 128, "int8")
    for b in (0, 5 * times + 2):
        cache.table[b] = fill
        cache.lens[b] = 0
    q = rounded(rng.standard_normal((sum(counts), 4, 128)), "bf16").cuda()
    out, lse = run_shared(cache, groups, q, counts, 0.1)
    check_attention(want, q, counts, 0.1, out, lse, None, None)
