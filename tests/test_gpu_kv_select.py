"""Selection of pages of the 8-bit key/value cache and attention over them, against plain
implementations (needs a GPU). Bounds and columns are whole numbers and compared exactly;
attention's tolerances are those of test_gpu_kv.py, over the selected tokens."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
import kv_select_reference as sel
import lossless_bit_level_gb300 as ibp
from kv_harness import as_float32, cache_of, offsets, pools, random_rows, rounded, with_lens
from test_gpu_kv import status_word

pytestmark = pytest.mark.gpu


def bounds_of(cache, fill=0x55):
    n, h, _, d = cache.k_codes.shape
    return torch.full((n, h, 2, d), fill, dtype=torch.int8, device="cuda")


def check_bounds(want, cache, bounds, begin, fill=0x55):
    """Pages from begin[b] on hold their bounds, the others what was there."""
    got, table = bounds.cpu().numpy(), cache.table.cpu().numpy()
    left = np.ones(got.shape[0], bool)
    for b, n in enumerate(want.lens):
        for j in range(max(begin[b], 0) // want.page, -(-n // want.page)):
            page = table[b, j]
            left[page] = False
            for h in range(want.heads):
                lo, hi = sel.bounds(want.tiles["k"][b][h][j][1], want.code)
                assert np.array_equal(got[page, h, 0], lo), (b, j, h)
                assert np.array_equal(got[page, h, 1], hi), (b, j, h)
    assert (got[left] == fill).all()


def select(cache, bounds, q, counts, pages, cu=True, status=None):
    max_q = max(counts, default=0)
    scratch = torch.empty(max(16, ibp.kv_select_scratch_bytes(cache)), dtype=torch.uint8,
                          device="cuda").fill_(0xFF)
    columns = torch.full((cache.batch, cache.n_heads, pages), -9, dtype=torch.int32, device="cuda")
    ibp.kv_select(cache, bounds, q, columns, scratch, cu_q=offsets(counts) if cu else None, max_q=max_q,
                  status=status)
    return columns


def attend(cache, columns, q, counts, scale, cu=True, status=None, out=None):
    n, heads, pages, max_q = q.shape[0], q.shape[1], columns.shape[2], max(counts, default=0)
    scratch = torch.empty(max(16, ibp.kv_attention_selected_scratch_bytes(cache, n, max_q, heads, pages)),
                          dtype=torch.uint8, device="cuda").fill_(0xFF)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((n, heads), 7.0, device="cuda")
    ibp.kv_attention_selected(cache, columns, q, out, scale, scratch, cu_q=offsets(counts) if cu else None,
                              max_q=max_q, lse=lse, status=status)
    return out, lse


def check_columns(want, q, counts, columns):
    got, qn, group, first = columns.cpu().numpy(), q.float().cpu().numpy(), q.shape[1] // want.heads, 0
    pages = got.shape[2]
    for b, n in enumerate(counts):
        for h in range(want.heads):
            rows = qn[first:first + n, h * group:(h + 1) * group].reshape(n * group, qn.shape[2])
            exp = sel.columns(want, b, h, rows, n, pages)
            assert got[b, h].tolist() == exp + [-1] * (pages - len(exp)), (b, h)
        first += n


def check_attention(want, q, counts, scale, columns, out, lse):
    group, first = q.shape[1] // want.heads, 0
    half = 2.0 ** (-8 if q.dtype == torch.bfloat16 else -11)
    qn, on, zn, cn = q.float().cpu().numpy(), out.float().cpu().numpy(), lse.cpu().numpy(), columns.cpu().numpy()
    for b, n in enumerate(counts):
        for h in range(want.heads):
            heads = slice(h * group, (h + 1) * group)
            o, z, size, spread = sel.attention(want, b, h, qn[first:first + n, heads],
                                               [c for c in cn[b, h] if c >= 0], scale)
            score = 2.0 ** -20 * spread + 2.0 ** -21
            tol = half * np.abs(o) * 1.01 + (2.0 ** -11 + 2 * score) * size + 2.0 ** -24
            assert (np.abs(on[first:first + n, heads] - o) <= tol).all(), (b, h)
            gz = zn[first:first + n, heads]
            assert np.array_equal(np.isneginf(gz), np.isneginf(z))
            ok = ~np.isneginf(z)
            assert (np.abs(gz[ok] - z[ok]) <= score + 2.0 ** -22 * np.abs(z[ok])).all()
        first += n


CASES = [
    # (lengths, query rows, q heads, kv heads, dim, page, code, dtype, pages)
    ([1], [1], 1, 1, 128, 16, "int8", "bf16", 2),
    ([0, 1, 16, 17, 33], [1, 1, 1, 1, 1], 4, 4, 64, 16, "int8", "fp16", 2),
    ([400, 64, 65, 0, 300], [1, 1, 1, 1, 1], 8, 2, 128, 16, "int8", "bf16", 5),
    ([900, 0, 31, 640], [1, 1, 1, 1], 10, 2, 128, 32, "e4m3", "bf16", 3),
    ([777, 1500], [1, 1], 16, 1, 128, 128, "e4m3", "fp16", 4),
    ([530, 5, 0, 333], [3, 7, 4, 0], 6, 2, 64, 16, "int8", "bf16", 9),
    ([2000, 90], [9, 40], 8, 4, 128, 64, "int8", "fp16", 6),
    ([700, 350, 257], [33, 20, 1], 8, 1, 64, 16, "e4m3", "bf16", 10),
    ([1100], [1], 128, 2, 64, 16, "int8", "bf16", 24),   # 64 shared heads: 64 rows
    ([1100, 420], [3, 2], 72, 2, 128, 32, "e4m3", "fp16", 7),  # 108 rows: two passes of 64
    ([300] * 3, [1] * 3, 4, 2, 64, 16, "int8", "bf16", 40),    # all pages fit
]


@pytest.mark.parametrize("lens,counts,q_heads,heads,dim,page,code,dtype,pages", CASES)
def test_bounds_selection_and_attention(lens, counts, q_heads, heads, dim, page, code, dtype, pages):
    rng = np.random.default_rng(sum(lens) + dim + pages)
    want = cache_of(rng, lens, heads, page, dim, code)
    cache, bounds, status = pools(want, rng), None, status_word()
    bounds = bounds_of(cache)
    ibp.kv_bounds(cache, bounds, status=status)
    check_bounds(want, cache, bounds, [0] * len(lens))
    q = rounded(1.5 * rng.standard_normal((sum(counts), q_heads, dim)), dtype).cuda()
    columns = select(cache, bounds, q, counts, pages, status=status)
    check_columns(want, q, counts, columns)
    scale = dim ** -0.5
    out, lse = attend(cache, columns, q, counts, scale, status=status)
    assert int(status.item()) == 0
    check_attention(want, q, counts, scale, columns, out, lse)


@pytest.mark.parametrize("lens,counts,q_heads,heads,dim,page,code,dtype,pages", CASES)
def test_selection_through_wide_tables(lens, counts, q_heads, heads, dim, page, code, dtype, pages):
    """Tables of more than 1024 columns, most of them unused: scores and choice in two kernels."""
    rng = np.random.default_rng(sum(lens) + dim + pages)
    want = cache_of(rng, lens, heads, page, dim, code)
    cache, status = pools(want, rng, cols=1100), status_word()
    bounds = bounds_of(cache)
    ibp.kv_bounds(cache, bounds, status=status)
    check_bounds(want, cache, bounds, [0] * len(lens))
    q = rounded(1.5 * rng.standard_normal((sum(counts), q_heads, dim)), dtype).cuda()
    columns = select(cache, bounds, q, counts, pages, status=status)
    assert int(status.item()) == 0
    check_columns(want, q, counts, columns)


def test_no_offsets_views_and_another_stream():
    rng = np.random.default_rng(2)
    want = cache_of(rng, [500, 260, 90], 2, 16, 64, "int8")
    cache = pools(want, rng)
    bounds = bounds_of(cache)
    stream, wide = torch.cuda.Stream(), rounded(rng.standard_normal((6, 9, 64)), "bf16").cuda()
    q, room = wide[:, 1:9:2], torch.zeros((6, 7, 64), dtype=torch.bfloat16, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ibp.kv_bounds(cache, bounds)
        columns = select(cache, bounds, q, [2, 2, 2], 6, cu=False)
        out, lse = attend(cache, columns, q, [2, 2, 2], 0.125, cu=False, out=room[:, 2:6])
    stream.synchronize()
    check_bounds(want, cache, bounds, [0, 0, 0])
    check_columns(want, q, [2, 2, 2], columns)
    check_attention(want, q, [2, 2, 2], 0.125, columns, out, lse)
    assert not room[:, :2].any() and not room[:, 6:].any()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_then_bounds_of_what_it_touched(code):
    """Decoding: after an append only the touched pages' bounds are brought up to date, also
    where the rows raised a page's scale and its codes moved."""
    rng = np.random.default_rng(3)
    lens, heads, page, dim = [30, 64, 5, 0], 2, 32, 128
    want = cache_of(rng, lens, heads, page, dim, code)
    cache = pools(want, rng, room=3 * page)
    bounds, begin, new_lens = bounds_of(cache), cache.lens.clone(), torch.empty_like(cache.lens)
    rows = random_rows(rng, 4 * 40, heads, dim)
    rows["k"] *= 30
    ibp.kv_append(cache, rows["k"].cuda(), rows["v"].cuda(), new_lens=new_lens)
    for b in range(4):
        want.append(b, as_float32({n: t[40 * b:40 * b + 40] for n, t in rows.items()}))
    after = with_lens(cache, new_lens)
    ibp.kv_bounds(after, bounds, begin=begin)
    check_bounds(want, after, bounds, lens)
    bounds = bounds_of(cache, 7)
    ibp.kv_bounds(after, bounds, begin=torch.tensor([-5, 70, 1000, 39], dtype=torch.int32, device="cuda"))
    check_bounds(want, after, bounds, [-5, 70, 1000, 39], 7)


def test_equal_scores_take_the_lowest_column():
    """Pages that are copies of one another, and rows of zeros: every score is the same."""
    rng = np.random.default_rng(4)
    want = ref.Cache(1, 1, 16, 64, "int8")
    one = as_float32(random_rows(rng, 16, 1, 64))
    for _ in range(40):
        want.append(0, one)
    cache = pools(want, rng)
    bounds = bounds_of(cache)
    ibp.kv_bounds(cache, bounds)
    for q in (rounded(rng.standard_normal((1, 4, 64)), "bf16"), torch.zeros((1, 4, 64), dtype=torch.bfloat16)):
        columns = select(cache, bounds, q.cuda(), [1], 9)
        assert columns[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 39]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_query_rows_that_are_odd(dtype):
    """Very small and very large rows, NaN and infinities in a row: the score's rule holds."""
    rng = np.random.default_rng(5)
    want = cache_of(rng, [640], 2, 16, 128, "e4m3")
    cache = pools(want, rng)
    bounds = bounds_of(cache)
    ibp.kv_bounds(cache, bounds)
    x = rng.standard_normal((8, 2, 128)).astype(np.float32)
    x[0] *= 2.0 ** -20 if dtype == "fp16" else 2.0 ** -120
    x[1] *= 2.0 ** 13 if dtype == "fp16" else 2.0 ** 110
    x[2, :, 5] = np.nan
    x[3, :, 7] = np.inf
    x[4, :, 9] = -np.inf
    x[5, :] = 0
    x[6, :, 1:] = 0
    for i in range(8):
        q = rounded(x[i:i + 1], dtype)
        check_columns(want, q, [1], select(cache, bounds, q.cuda(), [1], 7))


def test_many_pages_of_long_sequences():
    """More columns than one CTA keeps in shared memory (8192), against the same rule over the
    bounds in whole numbers."""
    H, P, D, n_tokens, pages = 2, 16, 64, 9001 * 16 + 5, 300
    g = torch.Generator(device="cuda").manual_seed(0)
    cols = -(-n_tokens // P)
    codes = torch.randint(-127, 128, (cols, H, P, D), generator=g, device="cuda", dtype=torch.int8)
    scales = torch.rand((cols, H), generator=g, device="cuda") + 0.5
    table = torch.randperm(cols, generator=g, device="cuda").to(torch.int32)[None]
    lens = torch.tensor([n_tokens], dtype=torch.int32, device="cuda")
    cache = ibp.KVCache(codes, codes, scales, scales, table, lens)
    bounds, status = bounds_of(cache), status_word()
    ibp.kv_bounds(cache, bounds, status=status)
    q = torch.randn((1, 2 * H, D), generator=g, device="cuda").bfloat16()
    columns = select(cache, bounds, q, [1], pages, status=status)
    assert int(status.item()) == 0
    at = table[0].long()
    x = codes[at].long()
    lo, hi = x.amin(2), x.amax(2)
    lo[-1], hi[-1] = x[-1, :, :5].amin(1), x[-1, :, :5].amax(1)
    for h in range(H):
        best = torch.full((cols,), -float("inf"), device="cuda", dtype=torch.float64)
        for r in range(2):
            n, e = sel.whole(q[0, 2 * h + r].float().cpu().numpy())
            n = torch.from_numpy(n).cuda()
            best = torch.maximum(best, torch.maximum(n * lo[:, h], n * hi[:, h]).sum(1).double() * 2.0 ** (e - 6))
        score = best.float() * scales[at, h]
        order = torch.sort(score[1:-1], descending=True, stable=True)[1][:pages - 2] + 1
        assert columns[0, h].tolist() == [0] + sorted(order.tolist()) + [cols - 1]
    again = select(cache, bounds, q, [1], pages)
    assert torch.equal(columns, again)


def test_lists_in_another_order_and_lists_that_are_wrong():
    rng = np.random.default_rng(6)
    want = cache_of(rng, [200, 150], 1, 16, 64, "int8")
    cache = pools(want, rng)
    q = rounded(rng.standard_normal((4, 2, 64)), "bf16").cuda()
    good = [[[5, 0, 9, 11, 12]], [[7, 2, 0, 4, 9]]]  # rows at 198, 199 and 148, 149

    def run(lists):
        status = status_word()
        columns = torch.tensor(lists, dtype=torch.int32, device="cuda")
        out, lse = attend(cache, columns, q, [2, 2], 0.125, status=status)
        return int(status.item()), columns, out, lse

    code, columns, out, lse = run(good)
    assert code == 0
    check_attention(want, q, [2, 2], 0.125, columns, out, lse)
    for entry, bad in ((0, -1), (0, 12), (1, 13), (4, 11), (4, -1), (0, 1 << 30), (2, -(1 << 31))):
        lists = [[list(good[0][0])], good[1]]
        lists[0][0][entry] = bad
        code, columns, out, lse = run(lists)
        assert code == ibp.ERR_INDEX
        # that page is left out, the other sequence is as it was
        kept = [c for i, c in enumerate(good[0][0]) if i != entry]
        columns = torch.tensor([[kept + [-1]], good[1]], dtype=torch.int32)
        check_attention(want, q, [2, 2], 0.125, columns, out, lse)


def test_bad_pages_are_reported():
    rng = np.random.default_rng(7)
    want = cache_of(rng, [200], 1, 16, 64, "int8")
    cache = pools(want, rng)
    bounds, q = bounds_of(cache), rounded(rng.standard_normal((1, 2, 64)), "bf16").cuda()
    ibp.kv_bounds(cache, bounds)
    cache.table[0, 3] = 10_000
    for call in (lambda s: ibp.kv_bounds(cache, bounds, status=s),
                 lambda s: select(cache, bounds, q, [1], 4, status=s)):
        status = status_word()
        call(status)
        assert int(status.item()) == ibp.ERR_INDEX
    # a page that is not there has the lowest score
    columns = select(cache, bounds, q, [1], 12)
    assert columns[0, 0].tolist() == [c for c in range(13) if c != 3]
    over = with_lens(cache, torch.tensor([99_999], dtype=torch.int32, device="cuda"))
    status = status_word()
    select(over, bounds, q, [1], 4, status=status)
    assert int(status.item()) == ibp.ERR_INDEX


def test_rows_of_no_sequence_are_left():
    rng = np.random.default_rng(8)
    want = cache_of(rng, [200, 90], 2, 16, 64, "int8")
    cache = pools(want, rng)
    bounds, q = bounds_of(cache), rounded(rng.standard_normal((9, 4, 64)), "fp16").cuda()
    ibp.kv_bounds(cache, bounds)
    cu = torch.tensor([2, 4, 6], dtype=torch.int32, device="cuda")
    scratch = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    columns = torch.zeros((2, 2, 4), dtype=torch.int32, device="cuda")
    ibp.kv_select(cache, bounds, q, columns, scratch, cu_q=cu, max_q=2)
    out = torch.full_like(q, 3.0)
    ibp.kv_attention_selected(cache, columns, q, out, 0.125, scratch, cu_q=cu, max_q=2)
    check_columns(want, q[2:6], [2, 2], columns)
    assert bool((out[:2] == 3).all()) and bool((out[6:] == 3).all())
    lse = torch.zeros((9, 4), device="cuda")
    ibp.kv_attention_selected(cache, columns, q, out, 0.125, scratch, cu_q=cu, max_q=2, lse=lse)
    check_attention(want, q[2:6], [2, 2], 0.125, columns, out[2:6], lse[2:6])


def test_two_graphs_replayed_in_turn():
    """A whole step captured: bounds, selection and attention, for two caches that share the
    workspace; replayed one after another with new queries, each as a plain call."""
    rng = np.random.default_rng(9)
    scratch = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    steps = []
    stream = torch.cuda.Stream()
    for code, lens in (("int8", [700, 40]), ("e4m3", [300, 900])):
        want = cache_of(rng, lens, 2, 16, 128, code)
        cache = pools(want, rng)
        bounds = bounds_of(cache)
        q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
        out, columns = torch.empty_like(q), torch.empty((2, 2, 6), dtype=torch.int32, device="cuda")
        lse = torch.empty((2, 8), device="cuda")

        def step(cache=cache, bounds=bounds, q=q, out=out, columns=columns, lse=lse):
            ibp.kv_bounds(cache, bounds)
            ibp.kv_select(cache, bounds, q, columns, scratch)
            ibp.kv_attention_selected(cache, columns, q, out, 0.1, scratch, lse=lse)

        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        steps.append((graph, want, q, out, columns, lse, step))  # (step holds the cache)
    for _ in range(3):
        for graph, want, q, out, columns, lse, _ in steps:
            q.copy_(rounded(rng.standard_normal((2, 8, 128)), "bf16"))
            graph.replay()
        torch.cuda.synchronize()
        for _, want, q, out, columns, lse, _ in steps:
            check_columns(want, q, [1, 1], columns)
            check_attention(want, q, [1, 1], 0.1, columns, out, lse)
