"""The 8-bit paged key/value cache on the GPU against plain 64-bit implementations
(needs a GPU).

Codes and scales follow a rule in single precision, so append, read and evict are
compared exactly. Attention's tolerances, per element, with A = sum_t p_t |v_t| and
X = the largest scale * sum_d |q_d k_d| of a row: the output is rounded once (half a
unit: 2^-8 of the value for bf16, 2^-11 for fp16) after probabilities of 11 bits
(2^-11 A at most, sums in 24 bits); a score carries at most 16 roundings of 2^-24 X
that do not cancel (accumulation in chunks, the scale, the exponential), so lse moves by
2^-20 X and probabilities by twice that, relatively."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
import lossless_bit_level_gb300 as ibp
from kv_harness import (DTYPES, as_float32, cache_of, offsets, pools, random_rows, read_all,
                        rounded, with_lens)

pytestmark = pytest.mark.gpu


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- append and read

APPENDS = [
    # (lengths before, rows each, heads, page, dim, code, dtype)
    ([0], [1], 1, 16, 64, "int8", "bf16"),
    ([0, 0, 0], [70, 1, 16], 3, 16, 128, "int8", "bf16"),
    ([5, 0, 64, 63, 65], [1, 1, 1, 1, 1], 2, 64, 128, "int8", "bf16"),
    ([5, 0, 64, 63, 65], [130, 0, 1, 2, 63], 2, 64, 128, "e4m3", "fp16"),
    ([31, 33], [40, 7], 5, 32, 64, "e4m3", "fp32"),
    ([100, 7, 128], [29, 300, 0], 2, 128, 128, "int8", "fp32"),
    ([17, 300], [0, 0], 2, 128, 64, "int8", "fp16"),
]


@pytest.mark.parametrize("lens,counts,heads,page,dim,code,dtype", APPENDS)
def test_append_is_exact(lens, counts, heads, page, dim, code, dtype):
    rng = np.random.default_rng(sum(lens) + sum(counts) + dim)
    want = cache_of(rng, lens, heads, page, dim, code, dtype)
    # room for the new rows: pages that hold nothing yet
    cache = pools(want, rng, room=max(counts) + page)
    rows = random_rows(rng, sum(counts), heads, dim, dtype)
    new_lens, status = torch.empty_like(cache.lens), status_word()
    cu = offsets(counts)
    k, v = rows["k"].cuda(), rows["v"].cuda()
    for _ in range(2):  # the second call leaves the pages as they are
        ibp.kv_append(cache, k, v, cu=cu, new_lens=new_lens, status=status)
    at = 0
    for b, n in enumerate(counts):
        if n:
            want.append(b, as_float32({m: t[at:at + n] for m, t in rows.items()}))
        at += n
    got = read_all(with_lens(cache, new_lens), max(want.lens) + 3)
    assert int(status.item()) == 0
    assert new_lens.tolist() == want.lens and cache.lens.tolist() == lens
    for name in "kv":
        for b in range(len(lens)):
            for h in range(heads):
                n = want.lens[b]
                assert np.array_equal(got[name][b, :n, h], want.values(name, b, h)), (name, b, h)
                assert not got[name][b, n:, h].any()


def test_append_uniform_strided_and_in_another_stream():
    """No offsets (the same count each), rows that are views of one fused tensor, a
    stream of their own."""
    rng = np.random.default_rng(4)
    lens, heads, page, dim, each = [3, 40, 0], 2, 32, 64, 37
    want = cache_of(rng, lens, heads, page, dim, "int8")
    cache = pools(want, rng, room=64)
    fused = torch.from_numpy(rng.standard_normal((3 * each, 7, dim)).astype(np.float32)).to(
        torch.bfloat16)
    new_lens, status = torch.empty_like(cache.lens), status_word()
    dev = fused.cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    ibp.kv_append(cache, dev[:, 1:5:2], dev[:, 5:7], new_lens=new_lens, status=status,
                  stream=stream)
    stream.synchronize()
    for b in range(3):
        part = fused[b * each:(b + 1) * each].float().numpy()
        want.append(b, {"k": part[:, 1:5:2], "v": part[:, 5:7]})
    got = read_all(with_lens(cache, new_lens), max(want.lens))
    assert int(status.item()) == 0
    for name in "kv":
        for b in range(3):
            for h in range(heads):
                assert np.array_equal(got[name][b, :want.lens[b], h], want.values(name, b, h))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_extreme_values(code):
    """Infinities, NaN, zeros, denormals, the largest floats; a page of zeros; a page
    whose later tokens need a larger scale."""
    big = np.float32(3.4028235e38)
    heads, page, dim = 1, 16, 64
    x = np.zeros((40, heads, dim), np.float32)
    x[0, 0, :6] = [np.inf, -np.inf, np.nan, 1.0, -0.0, 1e-42]
    x[16:32] = 0
    x[33, 0, 0], x[34, 0, 1] = big, -1.0
    want = ref.Cache(1, heads, page, dim, code)
    cache = pools(want, np.random.default_rng(1), room=48)
    new_lens, status = torch.empty_like(cache.lens), status_word()
    at = 0
    for n in (3, 13, 17, 1, 6):
        part = torch.from_numpy(x[at:at + n]).cuda()
        ibp.kv_append(cache, part, part.clone(), new_lens=new_lens, status=status)
        want.append(0, {"k": x[at:at + n], "v": x[at:at + n]})
        cache = with_lens(cache, new_lens.clone())
        at += n
    got = read_all(cache, 40)
    assert int(status.item()) == 0
    assert np.isfinite(got["k"]).all()
    assert np.array_equal(got["k"][0, :, 0], want.values("k", 0, 0))
    assert np.array_equal(got["v"][0, :, 0], want.values("v", 0, 0))


def test_read_window_and_dtypes():
    rng = np.random.default_rng(5)
    lens = [0, 1, 50, 129]
    want = cache_of(rng, lens, 2, 16, 128, "int8")
    cache = pools(want, rng)
    begin = torch.tensor([0, -3, 47, 100], dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        got = read_all(cache, 70, begin=begin, dtype=dtype)
        for b, n in enumerate(lens):
            for h in range(2):
                full = np.zeros((300, 128), np.float32)
                full[3:3 + n] = want.values("v", b, h)  # token t at row t + 3
                first = int(begin[b]) + 3
                exp = torch.from_numpy(full[first:first + 70].copy()).to(dtype).float().numpy()
                assert np.array_equal(got["v"][b, :, h], exp)
    only = torch.empty((4, 5, 2, 128), device="cuda")
    ibp.kv_read(cache, None, only)
    assert np.array_equal(only.cpu().numpy()[3, :, 1], want.values("v", 3, 1)[:5])


def test_bad_pages_lengths_and_offsets_are_reported():
    rng = np.random.default_rng(6)
    want = cache_of(rng, [40, 20], 2, 16, 64, "int8")
    cache = pools(want, rng, room=16)
    rows = random_rows(rng, 2, 2, 64)
    k, v = rows["k"].cuda(), rows["v"].cuda()
    q = torch.randn((2, 4, 64), device="cuda").bfloat16()

    def run(c, cu=None, finite=True):
        out = []
        scratch = torch.empty(ibp.kv_attention_scratch_bytes(c, 2, 2, 4, True), dtype=torch.uint8,
                              device="cuda")
        w = torch.zeros((2, 2, c.capacity), device="cuda")
        new = ibp.KVCache(*(t.clone() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)),
                          c.table.clone(), torch.zeros_like(c.lens))
        es = torch.empty(ibp.kv_evict_scratch_bytes(c, 30), dtype=torch.uint8, device="cuda")
        o = torch.empty_like(q)
        for call in (lambda s: ibp.kv_append(c, k, v, cu=cu, status=s),
                     lambda s: ibp.kv_read(c, torch.empty((2, 60, 2, 64), device="cuda"), None,
                                           status=s),
                     lambda s: ibp.kv_attention(c, q, o, 0.125, scratch, cu_q=cu,
                                                max_q=1 if cu is None else 2, weights=w,
                                                status=s),
                     lambda s: ibp.kv_evict(c, w, 30, 2, new, es, status=s)):
            st = status_word()
            call(st)
            torch.cuda.synchronize()
            out.append(int(st.item()))
        # a length past the capacity is clamped to it: slots that hold nothing are then used
        assert not finite or torch.isfinite(o.float()).all()
        return out

    bad = torch.tensor([cache.k_codes.shape[0], 5000], dtype=torch.int32, device="cuda")
    saved = cache.table.clone()
    cache.table[0, 2], cache.table[1, 1] = bad[0], -7
    assert run(cache) == [ibp.ERR_INDEX] * 4
    cache.table.copy_(saved)
    assert run(with_lens(cache, torch.tensor([40, 5000], dtype=torch.int32, device="cuda")),
               finite=False) == [ibp.ERR_INDEX] * 4
    assert run(with_lens(cache, torch.tensor([-1, 20], dtype=torch.int32, device="cuda"))) == \
        [ibp.ERR_INDEX] * 4
    cu = torch.tensor([0, 5, 2], dtype=torch.int32, device="cuda")
    got = run(cache, cu)
    assert got[0] == got[2] == ibp.ERR_INDEX


# ---------------------------------------------------------------- attention

def run_attention(cache, q, counts, scale, weights=True, cu=True, lse=True, decay=0.5, seed=0,
                  out=None, stream=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, heads = q.shape[0], q.shape[1]
    max_q = max(counts, default=0)
    scratch = torch.empty(max(16, ibp.kv_attention_scratch_bytes(cache, n, max_q, heads, weights)),
                          dtype=torch.uint8, device="cuda").fill_(0xFF)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    z = torch.full((n, heads), 7.0, device="cuda") if lse else None
    w_in = w = None
    if weights:
        shape = (cache.batch, cache.n_heads, cache.capacity + 5)
        w_in = torch.rand(shape, generator=g, device="cuda")
        w = torch.full(shape, -3.0, device="cuda")
    status = status_word()
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    ibp.kv_attention(cache, q, out, scale, scratch, cu_q=offsets(counts) if cu else None,
                     max_q=max_q, lse=z, weights=w, weights_in=w_in, decay=decay, status=status,
                     stream=stream)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, z, w, w_in


def check_attention(want, q, counts, scale, out, lse, w, w_in, decay=0.5):
    heads = q.shape[1]
    group, first = heads // want.heads, 0
    half = 2.0 ** (-8 if q.dtype == torch.bfloat16 else -11)
    qn, on = q.float().cpu().numpy(), out.float().cpu().numpy()
    zn = None if lse is None else lse.cpu().numpy()
    for b, n in enumerate(counts):
        for h in range(want.heads):
            k = want.values("k", b, h).astype(np.float64)
            v = want.values("v", b, h).astype(np.float64)
            mine = qn[first:first + n, h * group:(h + 1) * group]
            o, z, p = ref.attention(mine, k, v, scale)
            size, _, _ = ref.attention(mine, k, np.abs(v), scale)
            spread = scale * (np.abs(mine).reshape(n * group, q.shape[2]) @ np.abs(k).T).max(
                initial=0.0)
            score = 2.0 ** -20 * spread + 2.0 ** -21
            tol = half * np.abs(o) * 1.01 + (2.0 ** -11 + 2 * score) * size + 2.0 ** -24
            got = on[first:first + n, h * group:(h + 1) * group]
            assert (np.abs(got - o) <= tol).all(), (b, h, np.abs(got - o).max())
            if zn is not None:
                gz = zn[first:first + n, h * group:(h + 1) * group]
                assert np.array_equal(np.isneginf(gz), np.isneginf(z))
                ok = ~np.isneginf(z)
                assert (np.abs(gz[ok] - z[ok]) <= score + 2.0 ** -22 * np.abs(z[ok])).all()
            if w is not None:
                t = want.lens[b]
                gw, gi = w[b, h].cpu().numpy(), w_in[b, h].cpu().numpy().astype(np.float64)
                exp = decay * gi[:t] + p
                assert (np.abs(gw[:t] - exp) <= 2.0 ** -22 * exp + 2 * score * p + 1e-30).all()
                assert (gw[t:] == -3.0).all()  # entries past the length are left alone
        first += n


ATTENDS = [
    # (lengths, query rows, q heads, kv heads, dim, page, code, dtype)
    ([1], [1], 1, 1, 128, 16, "int8", "bf16"),
    ([0, 1, 2, 17], [1, 1, 1, 1], 4, 4, 64, 16, "int8", "fp16"),
    ([63, 64, 65, 0, 300], [1, 1, 1, 1, 1], 8, 2, 128, 64, "int8", "bf16"),
    ([63, 64, 65, 0, 300], [1, 1, 1, 1, 1], 10, 2, 128, 32, "e4m3", "bf16"),
    ([777, 1500], [1, 1], 16, 1, 128, 128, "e4m3", "fp16"),
    ([130, 5, 0, 33], [3, 7, 4, 0], 6, 2, 64, 16, "int8", "bf16"),
    ([200, 90], [9, 40], 8, 4, 128, 64, "int8", "fp16"),
    ([200, 90, 257], [33, 90, 1], 8, 1, 64, 32, "e4m3", "bf16"),
    ([300, 129], [300, 60], 4, 2, 128, 64, "int8", "bf16"),
    ([513], [200], 8, 1, 128, 16, "e4m3", "fp16"),
    ([4097], [1], 32, 8, 128, 64, "int8", "bf16"),
]


@pytest.mark.parametrize("lens,counts,q_heads,heads,dim,page,code,dtype", ATTENDS)
@pytest.mark.parametrize("weights", [False, True])
def test_attention(lens, counts, q_heads, heads, dim, page, code, dtype, weights):
    rng = np.random.default_rng(sum(lens) + 7 * sum(counts) + dim)
    want = cache_of(rng, lens, heads, page, dim, code)
    cache = pools(want, rng)
    q = rounded(1.5 * rng.standard_normal((sum(counts), q_heads, dim)), dtype).cuda()
    scale = 1.0 / np.sqrt(dim)
    out, lse, w, w_in = run_attention(cache, q, counts, scale, weights)
    check_attention(want, q, counts, scale, out, lse, w, w_in)
    again = run_attention(cache, q, counts, scale, weights)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    if weights:
        assert torch.equal(w, again[2])


def test_attention_strides_streams_and_no_offsets():
    """Rows that are views of fused tensors, the same count each, no lse; a stream of its
    own; weights accumulated in place."""
    rng = np.random.default_rng(11)
    lens, heads, q_heads, dim, each = [70, 5, 129], 2, 4, 64, 2
    want = cache_of(rng, lens, heads, 32, dim, "int8")
    cache = pools(want, rng)
    fused = rounded(rng.standard_normal((6, 9, dim)), "bf16").cuda()
    q = fused[:, 1:9:2]
    out = torch.zeros((6, 12, dim), dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    got, _, w, w_in = run_attention(cache, q, [each] * 3, 0.1, cu=False, lse=False,
                                    out=out[:, 2:10:2], stream=stream)
    check_attention(want, q, [each] * 3, 0.1, got, None, w, w_in)
    assert not out[:, 0].any() and not out[:, 3].any() and not out[:, 10:].any()
    acc = w_in.clone()
    scratch = torch.empty(ibp.kv_attention_scratch_bytes(cache, 6, 2, q_heads, True),
                          dtype=torch.uint8, device="cuda")
    ibp.kv_attention(cache, q, torch.empty_like(q), 0.1, scratch, max_q=2, weights=acc,
                     weights_in=acc, decay=0.5)
    for b, n in enumerate(lens):
        assert torch.equal(acc[b, :, :n], w[b, :, :n])


def test_attention_large_scores_and_value_scales():
    """Scores of hundreds, values of very different size from page to page (a page of
    zeros among them), a negative scale: nothing overflows and nothing is lost."""
    rng = np.random.default_rng(12)
    heads, dim, page = 1, 64, 16
    want = ref.Cache(1, heads, page, dim, "int8")
    for j, f in enumerate([1.0, 1e-12, 1e15, 0.0, 1e-25, 3.0, 1e4]):
        x = rng.standard_normal((page, heads, dim)).astype(np.float32)
        want.append(0, {"k": 6 * x, "v": (f * rng.standard_normal((page, heads, dim))).astype(
            np.float32)})
    cache = pools(want, rng)
    for scale, gain in ((1.0, 6.0), (-0.3, 2.0), (0.0, 1.0)):
        q = rounded(gain * rng.standard_normal((3, 2, dim)), "bf16").cuda()
        out, lse, w, w_in = run_attention(cache, q, [3], scale)
        k, v = want.values("k", 0, 0), want.values("v", 0, 0)
        o, z, p = ref.attention(q.float().cpu().numpy(), k, v, scale)
        size, _, _ = ref.attention(q.float().cpu().numpy(), k, np.abs(v), scale)
        spread = abs(scale) * (np.abs(q.float().cpu().numpy()).reshape(6, dim) @ np.abs(k).T).max()
        score = 2.0 ** -20 * spread + 2.0 ** -21
        tol = 2.0 ** -8 * 1.01 * np.abs(o) + (2.0 ** -11 + 2 * score) * size + 2.0 ** -24
        assert (np.abs(out.float().cpu().numpy() - o) <= tol).all()
        assert (np.abs(lse.cpu().numpy() - z) <= score + 2.0 ** -22 * np.abs(z)).all()
        gi = w_in[0, 0, :112].cpu().numpy().astype(np.float64)
        assert (np.abs(w[0, 0, :112].cpu().numpy() - (0.5 * gi + p)) <=
                2.0 ** -22 * (0.5 * gi + p) + 2 * score * p + 1e-30).all()


def test_attention_query_magnitudes():
    """bf16 query rows far outside fp16's range, large and small in one call."""
    rng = np.random.default_rng(13)
    lens = [90]
    want = cache_of(rng, lens, 1, 16, 64, "int8")
    cache = pools(want, rng)
    x = rng.standard_normal((4, 2, 64)) * np.array([1e30, 1e-30, 1.0, 3e5])[:, None, None]
    q = rounded(x, "bf16").cuda()
    for i, scale in enumerate((1e-31, 1e29, 0.1, 1e-6)):
        row = q[i:i + 1].contiguous()
        out, lse, _, _ = run_attention(cache, row, [1], scale, weights=False)
        check_attention(want, row, [1], scale, out, lse, None, None)


def test_attention_in_a_graph_and_pages_past_4_gib():
    """Captured and replayed with other lengths; pages whose bytes lie past 2^32."""
    heads, page, dim = 32, 128, 128
    n_pages = 8300  # 512 KiB a page: the last ones start past 4 GiB
    rng = np.random.default_rng(14)
    one = cache_of(rng, [300], 1, page, dim, "int8")
    k = torch.zeros((n_pages, heads, page, dim), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = (torch.zeros((n_pages, heads), device="cuda") for _ in range(2))
    ids = [8299, 8250, 8222]
    for j, page_id in enumerate(ids):
        for name, codes, scales in (("k", k, ks), ("v", v, vs)):
            s, c = one.tiles[name][0][0][j]
            codes[page_id, 31, :len(c)] = torch.from_numpy(c.astype(np.int8)).cuda()
            scales[page_id, 31] = float(s)
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    cache = ibp.KVCache(k, v, ks, vs, table, lens)
    got = read_all(cache, 300)
    assert np.array_equal(got["v"][0, :, 31], one.values("v", 0, 0))
    q = rounded(rng.standard_normal((1, heads, dim)), "bf16").cuda()
    out, status = torch.empty_like(q), status_word()
    scratch = torch.empty(ibp.kv_attention_scratch_bytes(cache, 1, 1, heads, False),
                          dtype=torch.uint8, device="cuda")
    ibp.kv_attention(cache, q, out, 0.1, scratch, status=status)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ibp.kv_attention(cache, q, out, 0.1, scratch, status=status)
    for n in (300, 257, 1, 0):
        lens.fill_(n)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        o, _, _ = ref.attention(q[:, 31:].float().cpu().numpy(), one.values("k", 0, 0, n),
                                one.values("v", 0, 0, n), 0.1)
        assert np.abs(out[0, 31].float().cpu().numpy() - o[0, 0]).max() <= 2.0 ** -8 * max(
            1e-6, np.abs(o).max()) + 2.0 ** -11 * np.abs(one.values("v", 0, 0)).max()
    assert int(status.item()) == 0
    # rows appended to the far page
    lens.fill_(300)
    rows = random_rows(rng, 5, heads, dim)
    new_lens = torch.empty_like(lens)
    ibp.kv_append(cache, rows["k"].cuda(), rows["v"].cuda(), new_lens=new_lens)
    one.append(0, {n: t[:, 31:].float().numpy() for n, t in rows.items()})
    got = read_all(with_lens(cache, new_lens), 305)
    assert np.array_equal(got["k"][0, :, 31], one.values("k", 0, 0))


# ---------------------------------------------------------------- eviction

EVICTS = [
    # (lengths, heads, page, dim, code, budget, recent, kind of weights)
    ([1], 1, 16, 64, "int8", 1, 0, "random"),
    ([0, 40, 41, 300], 2, 16, 64, "int8", 40, 8, "random"),
    ([1500, 64, 129], 3, 64, 128, "int8", 65, 64, "random"),
    ([1500, 2100], 2, 32, 128, "e4m3", 1024, 0, "random"),
    ([700, 90], 2, 128, 64, "e4m3", 77, 77, "random"),
    ([3000], 1, 64, 64, "int8", 1300, 100, "ties"),
    ([500], 2, 16, 64, "int8", 100, 3, "equal"),
    ([2500, 50], 1, 16, 128, "int8", 333, 10, "odd"),
]


def weights_like(rng, kind, n):
    if kind == "equal":
        return np.zeros(n, np.float32)
    if kind == "ties":
        return rng.integers(0, 5, n).astype(np.float32)
    w = (rng.random(n) ** 8).astype(np.float32)
    if kind == "odd" and n:
        w[rng.integers(0, n, n // 3)] = rng.choice(
            np.array([np.nan, -0.0, 0.0, np.inf, -np.inf, -1.0, 1e-42], np.float32), n // 3)
    return w


@pytest.mark.parametrize("lens,heads,page,dim,code,budget,recent,kind", EVICTS)
def test_evict_is_exact(lens, heads, page, dim, code, budget, recent, kind):
    rng = np.random.default_rng(sum(lens) + budget)
    src = cache_of(rng, lens, heads, page, dim, code)
    cache = pools(src, rng)
    w = [[weights_like(rng, kind, n) for _ in range(heads)] for n in lens]
    wt = np.full((len(lens), heads, cache.capacity + 3), np.nan, np.float32)
    for b, n in enumerate(lens):
        for h in range(heads):
            wt[b, h, :n] = w[b][h]
    want, kept = src.evict(w, budget, recent)
    empty = ref.Cache(len(lens), heads, page, dim, code)
    dst = pools(empty, rng, room=budget)
    scratch = torch.empty(ibp.kv_evict_scratch_bytes(cache, budget), dtype=torch.uint8,
                          device="cuda")
    new_w = torch.full((len(lens), heads, budget + 2), 5.0, device="cuda")
    keep = torch.full((len(lens), heads, budget), 5, dtype=torch.int32, device="cuda")
    status = status_word()
    ibp.kv_evict(cache, torch.from_numpy(wt).cuda(), budget, recent, dst, scratch,
                 new_weights=new_w, kept=keep, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert dst.lens.tolist() == want.lens
    got = read_all(dst, budget)
    for b, n in enumerate(want.lens):
        for h in range(heads):
            assert keep[b, h, :n].tolist() == kept[b][h].tolist()
            assert (keep[b, h, n:] == -1).all()
            assert np.array_equal(new_w[b, h, :n].cpu().numpy(), w[b][h][kept[b][h]],
                                  equal_nan=True)
            assert not new_w[b, h, n:].any()
            for name in "kv":
                assert np.array_equal(got[name][b, :n, h], want.values(name, b, h))
