"""Bounds, selection of pages and attention over them where numbers or sizes are odd (needs a GPU):
query rows with whole runs of NaN, codes and rows that are not finite, more sequences than one launch
is for. Bounds and columns are compared exactly; tolerances are those of test_gpu_kv_select.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
import kv_select_reference as sel
import lossless_bit_level_gb300 as ibp
from kv_harness import TORCH_CODE, cache_of, offsets, pools, rounded
from test_gpu_kv import status_word
from test_gpu_kv_select import attend, bounds_of, check_attention, check_bounds, check_columns, select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [None, 1100])  # one kernel, and two
@pytest.mark.parametrize("rows,group,dim", [(1, 4, 128), (2, 4, 64), (3, 5, 64), (9, 12, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows_with_runs_of_nan(dtype, rows, group, dim, cols):
    """A NaN counts as 0 wherever it stands, also where it has neighbours: the row's other elements
    set its exponent, and with it what the rows beside it are compared to."""
    rng = np.random.default_rng(rows + group + dim)
    heads = 2
    want = cache_of(rng, [700, 333], heads, 16, dim, "int8")
    cache, status = pools(want, rng, cols=cols), status_word()
    bounds = bounds_of(cache)
    ibp.kv_bounds(cache, bounds, status=status)
    x = rng.standard_normal((2 * rows, heads * group, dim)).astype(np.float32)
    for start, run in ((0, 4), (8, 4), (dim - 4, 4), (1, 11), (0, dim - 5), (0, dim)):
        y = x.copy()
        odd = [rows // 2, rows]  # a row of each sequence
        y[odd, 1::group] *= 20  # larger than those beside it: it chooses the pages
        y[odd, 1::group, start:start + run] = np.nan
        if run == 11:
            y[odd, 1::group, start:start + run:3] = -np.nan
        q = rounded(y, dtype)
        columns = select(cache, bounds, q.cuda(), [rows, rows], 7, status=status)
        check_columns(want, q, [rows, rows], columns)
    assert int(status.item()) == 0


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_bounds_of_codes_that_no_append_writes(code):
    """A NaN code counts as the largest number of its sign, -128 as -127; also as a page's only ones."""
    g = torch.Generator().manual_seed(3)
    n_pages, heads, page, dim, length = 9, 2, 32, 64, 7 * 32 + 5
    raw = torch.randint(0, 256, (n_pages, heads, page, dim), generator=g, dtype=torch.uint8)
    raw[1], raw[2] = 0x7F, 0xFF  # (int8: 127 and -1)
    raw[3] = 0x80                # (e4m3: -0)
    raw[4, :, ::2] = 0x7F
    raw[4, :, 1::2] = 0xFF
    codes = raw.cuda().view(TORCH_CODE[code])
    scales = torch.ones((n_pages, heads), device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None].contiguous()
    cache = ibp.KVCache(codes, codes, scales, scales, table, torch.tensor([length], dtype=torch.int32, device="cuda"))
    bounds, status = bounds_of(cache), status_word()
    ibp.kv_bounds(cache, bounds, status=status)
    assert int(status.item()) == 0
    x = ref.decode(raw.numpy(), code)
    if code == "e4m3":
        x = np.where(np.isnan(x), np.where(raw.numpy() & 0x80, -448.0, 448.0), x)
    got = bounds.cpu().numpy()
    for j in range(8):
        held = min(length - j * page, page)
        for h in range(heads):
            lo, hi = sel.bounds(x[j, h, :held], code)
            assert np.array_equal(got[j, h, 0], lo) and np.array_equal(got[j, h, 1], hi), (j, h)
    assert (got[8] == 0x55).all()


@pytest.mark.parametrize("n,group", [(1, 2), (3, 4), (20, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_rows_that_are_not_finite_over_lists(n, group, dtype, value):
    """One element of one row and head is not finite: with a NaN that row's output is NaN and its sum
    that of a row without tokens, as undivided, and every other row's is right."""
    rng = np.random.default_rng(n)
    dim, heads, counts = 64, 2, [n, n]
    want = cache_of(rng, [900, 270], heads, 16, dim, "int8")
    cache = pools(want, rng)
    x = rng.standard_normal((2 * n, heads * group, dim)).astype(np.float32)
    columns = torch.full((2, heads, 8), -1, dtype=torch.int32)
    for b, length in enumerate((900, 270)):
        own = list(range((length - n) // 16, -(-length // 16)))
        for h in range(heads):
            some = sorted(rng.choice(own[0], 8 - len(own), replace=False).tolist())
            columns[b, h] = torch.tensor(some + own)
    columns = columns.cuda()
    row, head = n // 2, group  # of the second K/V head
    x[row, head, 7] = value
    out, lse = attend(cache, columns, rounded(x, dtype).cuda(), counts, 0.125)
    if np.isnan(value):
        assert torch.isnan(out[row, head]).all() and lse[row, head] == -np.inf
    x[row, head] = 0
    q = rounded(x, dtype).cuda()
    clean, clean_lse = attend(cache, columns, q, counts, 0.125)
    out[row, head], lse[row, head] = clean[row, head], clean_lse[row, head]
    check_attention(want, q, counts, 0.125, columns, out, lse)


@pytest.mark.parametrize("cols", [None, 1100])  # selection in one kernel, and in two
def test_more_sequences_than_a_launch_is_for(cols):
    """1,100 short sequences, empty ones and ones without rows among them: bounds and selection go in
    slabs of 1,024, attention in slabs of 256 that share a workspace; as calls and captured."""
    rng = np.random.default_rng(11)
    batch, heads, page, dim, pages = 1100, 2, 16, 64, 4
    lens = [int(t) for t in rng.integers(0, 150, batch)]
    for b in (0, 255, 256, 1023, 1024, 1099):
        lens[b] = 140
    lens[1], lens[1025] = 0, 0
    counts = [int(t) for t in rng.integers(0, 3, batch)]
    for b in (255, 256, 1023, 1024):
        counts[b] = 2
    want = cache_of(rng, lens, heads, page, dim, "int8")
    cache, status = pools(want, rng, cols=cols), status_word()
    begin = [int(t) for t in rng.integers(-3, 150, batch)]
    bounds = bounds_of(cache, 7)
    ibp.kv_bounds(cache, bounds, begin=torch.tensor(begin, dtype=torch.int32, device="cuda"), status=status)
    check_bounds(want, cache, bounds, begin, 7)
    bounds = bounds_of(cache)
    ibp.kv_bounds(cache, bounds, status=status)
    check_bounds(want, cache, bounds, [0] * batch)
    q = rounded(1.5 * rng.standard_normal((sum(counts), 2 * heads, dim)), "bf16").cuda()
    columns = select(cache, bounds, q, counts, pages, status=status)
    check_columns(want, q, counts, columns)
    out, lse = attend(cache, columns, q, counts, 0.125, status=status)
    assert int(status.item()) == 0
    check_attention(want, q, counts, 0.125, columns, out, lse)
    # the whole step as a graph, over other queries first
    cu, n = offsets(counts), q.shape[0]
    scratch = torch.empty(max(ibp.kv_select_scratch_bytes(cache),
                              ibp.kv_attention_selected_scratch_bytes(cache, n, 2, 2 * heads, pages)),
                          dtype=torch.uint8, device="cuda")
    q2, columns2, out2, lse2 = (torch.empty_like(t) for t in (q, columns, out, lse))
    bounds2 = torch.empty_like(bounds)

    def step():
        ibp.kv_bounds(cache, bounds2)
        ibp.kv_select(cache, bounds2, q2, columns2, scratch, cu_q=cu, max_q=2)
        ibp.kv_attention_selected(cache, columns2, q2, out2, 0.125, scratch, cu_q=cu, max_q=2, lse=lse2)

    q2.copy_(q.flip(0))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()
    q2.copy_(q)
    for _ in range(3):
        for t in (columns2, out2, lse2):
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((columns, columns2), (out, out2), (lse, lse2)):
            assert torch.equal(a, b)
