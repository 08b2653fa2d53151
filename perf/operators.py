"""What the 8-bit key/value cache operators are measured on.

The operators: rows of keys and values put into a paged cache that holds 8 bits an
element with one scale for each page and head (append), the rows read back as values
(read), attention over that cache with its per-token sums of probabilities
(attention), and eviction of the tokens that were attended least, the kept ones
requantised into new pages (evict).

A cache: codes [pages, heads, page_tokens, head_dim] (int8 or float8 e4m3) and scales
[pages, heads] for keys and for values, a page table [batch, columns] (-1: no page) and
lengths [batch]. Token t of sequence b lies in slot t % page_tokens of page
table[b, t // page_tokens]; its value is code * scale.

Quantising a page whose largest finite magnitude is a: scale = a / qmax (qmax 127 for
int8, 448 for e4m3) held in [2^-100, 2^120], 0 where a is 0; code = the value times
1/scale, rounded to nearest even and saturated. Tokens appended to a page that is partly
filled raise its scale where they need to (never lower it), and the codes that are there
are then rescaled by old scale / new scale and rounded again.
"""
import math
import random

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
TORCH_CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
SMALLEST, LARGEST = 2.0 ** -100, 2.0 ** 120


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one short conversation, one query token: a call whose latency is what counts
        dict(name="attend one", op="attend", batch=1, q_heads=32, kv_heads=8, head_dim=128, page=16,
             code="int8", dtype="bf16", longest=777, shortest=777, queries=1, even=True, weights=False),
        # the K and V cache of one decoder layer as this repository stores it (8 x 4096 tokens,
        # 32 heads of 128, no shared heads), one token a sequence, weights for a later eviction
        dict(name="attend layer", op="attend", batch=8, q_heads=32, kv_heads=32, head_dim=128, page=64,
             code="int8", dtype="bf16", longest=4096, shortest=4096, queries=1, even=True, weights=True),
        # two long documents of different lengths with shared heads: few rows, a long axis
        dict(name="attend long", op="attend", batch=2, q_heads=32, kv_heads=8, head_dim=128, page=64,
             code="e4m3", dtype="bf16", longest=120_001, shortest=70_000, queries=1, even=True,
             weights=False),
        # a ragged batch (an empty sequence among it) that checks a few proposed tokens a sequence
        dict(name="attend verify", op="attend", batch=48, q_heads=16, kv_heads=4, head_dim=64, page=32,
             code="int8", dtype="fp16", longest=7_003, shortest=0, queries=7, even=False, weights=True),
        # a prompt fed in chunks: many query rows against the cache so far, bound by arithmetic
        dict(name="attend chunk", op="attend", batch=2, q_heads=32, kv_heads=8, head_dim=128, page=64,
             code="int8", dtype="bf16", longest=8_192, shortest=5_001, queries=2_048, even=False,
             weights=False),
        # one new token for each of a batch of conversations
        dict(name="append tokens", op="append", batch=64, kv_heads=8, head_dim=128, page=64, code="int8",
             dtype="bf16", longest=4_000, shortest=1, rows=1, even=True),
        # the whole prompts of one decoder layer in this repository's size
        dict(name="append layer", op="append", batch=8, kv_heads=32, head_dim=128, page=64, code="int8",
             dtype="bf16", longest=0, shortest=0, rows=4_096, even=True),
        # ragged pieces of prompts in 32 bits, behind pages that are partly filled
        dict(name="append pieces", op="append", batch=21, kv_heads=8, head_dim=64, page=16, code="e4m3",
             dtype="fp32", longest=1_501, shortest=3, rows=333, even=False),
        # a short conversation that went a little over its budget
        dict(name="evict few", op="evict", batch=1, kv_heads=8, head_dim=128, page=16, code="int8",
             dtype="bf16", longest=700, shortest=700, budget=512, recent=128),
        # one decoder layer's cache halved
        dict(name="evict layer", op="evict", batch=8, kv_heads=32, head_dim=128, page=64, code="int8",
             dtype="bf16", longest=4_096, shortest=1_900, budget=2_048, recent=256),
        # long documents cut down hard
        dict(name="evict long", op="evict", batch=2, kv_heads=8, head_dim=128, page=64, code="e4m3",
             dtype="bf16", longest=100_003, shortest=61_000, budget=12_345, recent=1_024),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        # no more than the largest listed cases: bytes moved, operations, and elements held
        if c["op"] == "attend":
            held = c["batch"] * c["kv_heads"] * c["head_dim"] * c["longest"]
            scores = c["batch"] * c["q_heads"] * c["queries"] * c["longest"]
            if w["bytes"] <= 4.2e8 and w["flops"] <= 3.5e11 and held <= 2.5e8 and scores <= 1.0e9:
                return c
        elif w["bytes"] <= (1.3e9 if c["op"] == "append" else 4.5e8):
            held = c["batch"] * c["kv_heads"] * c["head_dim"] * (c["longest"] + c.get("rows", 0))
            if held <= 2.1e8:
                return c


def _draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    batch = _log(rng, 1, 64)
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    c = dict(op=op, batch=batch, kv_heads=kv_heads, head_dim=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128]), code=rng.choice(["int8", "int8", "e4m3"]))
    longest = _log(rng, 1, 120_000)
    shortest = min(longest, rng.choice([0, 1, longest // 3, longest]))
    if op == "attend":
        group = rng.choice([1, 2, 4, 8, 5])
        queries = rng.choice([1, 1, _log(rng, 1, 16), _log(rng, 1, 2048)])
        c.update(dtype=rng.choice(["bf16", "fp16"]), q_heads=kv_heads * group, longest=longest,
                 shortest=shortest, queries=min(queries, max(longest, 1)), even=rng.random() < 0.5,
                 weights=queries <= 16 and rng.random() < 0.5)
    elif op == "append":
        c.update(dtype=rng.choice(["bf16", "fp16", "fp32"]), longest=rng.choice([0, min(longest, 8_000)]),
                 rows=rng.choice([1, _log(rng, 1, 4_096)]), even=rng.random() < 0.5)
        c["shortest"] = min(c["longest"], shortest)
    else:
        budget = _log(rng, 1, 16_384)
        c.update(dtype=rng.choice(["bf16", "fp16", "fp32"]), longest=longest, shortest=shortest,
                 budget=budget, recent=rng.choice([0, 1, budget // 8, budget // 2]))
    return c


# ------------------------------------------- sizes that follow from a case alone

def _spread(low, high, n):
    """n whole numbers from high down to low, spread as a low-discrepancy sequence."""
    if n == 1:
        return [high]
    return [high, low] + [low + int((high - low + 1) * ((0.6180339887 * i) % 1.0)) for i in range(1, n - 1)]


def _lengths(c):
    return _spread(c["shortest"], c["longest"], c["batch"])


def _counts(c):
    """New rows (append) or query rows (attend) of each sequence."""
    most = c["rows"] if c["op"] == "append" else c["queries"]
    return [most] * c["batch"] if c["even"] else _spread(1, most, c["batch"])


def _pages(n, page):
    return -(-n // page)


def work(case):
    c = case
    H, D, P = c["kv_heads"], c["head_dim"], c["page"]
    lens = _lengths(c)
    if c["op"] == "attend":
        counts = _counts(c)
        n, Hq = sum(counts), c["q_heads"]
        nbytes = sum(2 * t * H * D + 8 * _pages(t, P) * H for t in lens)
        nbytes += 2 * n * Hq * D * SIZE[c["dtype"]] + 4 * n * Hq
        if c["weights"]:
            nbytes += 8 * H * sum(lens)
        pairs = sum(sum(max(0, t - m + i + 1) for i in range(m)) for t, m in zip(lens, counts))
        return {"bytes": nbytes, "flops": 4 * Hq * D * pairs}
    if c["op"] == "append":
        counts = _counts(c)
        n, out = sum(counts), SIZE[c["dtype"]]
        window = _window(c) * P * c["batch"]
        # rows read, their codes written, the touched pages' values written
        return {"bytes": 2 * H * D * (n * SIZE[c["dtype"]] + n + window * out), "flops": 6 * 2 * H * D * n}
    kept = [min(t, c["budget"]) for t in lens]
    out = SIZE[c["dtype"]]
    # weights read; kept codes read and written; their values, weights and indices written
    nbytes = 4 * H * sum(lens) + 2 * H * D * 2 * sum(kept)
    nbytes += c["batch"] * c["budget"] * H * (2 * D * out + 8)
    return {"bytes": nbytes, "flops": 6 * 2 * H * D * sum(kept)}


def _window(c):
    """Pages that the new rows of one sequence touch, at most."""
    P = c["page"]
    return max(_pages(t + m, P) - t // P for t, m in zip(_lengths(c), _counts(c)))


# ---------------------------------------------------------------- inputs

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _channels(shape, g, device):
    """Keys and values are normal, with about 1% of the channels ten times as large."""
    x = torch.ones(shape, device=device)
    return torch.where(torch.rand(shape, generator=g, device=device) < 0.01, 10.0 * x, x)


def _quantised(n_pages, c, g, device):
    """Pages as an earlier append left them: every slot holds something."""
    H, P, D = c["kv_heads"], c["page"], c["head_dim"]
    x = torch.randn((n_pages, H, P, D), generator=g, device=device)
    x *= _channels((1, H, 1, D), g, device)
    s = x.abs().amax((2, 3)) / QMAX[c["code"]]
    x /= s[:, :, None, None]
    code = x.round_().to(torch.int8) if c["code"] == "int8" else x.to(torch.float8_e4m3fn)
    return code, s


def _paged(c, tokens, capacity, g, device):
    """A page table with pages in random order for `tokens` of each sequence, and the number of pages."""
    P = c["page"]
    need = [_pages(t, P) for t in tokens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=device).to(torch.int32)
    cols = max(1, _pages(capacity, P))
    start = torch.tensor([sum(need[:b]) for b in range(len(need))], device=device)
    j = torch.arange(cols, device=device)
    used = j[None, :] < torch.tensor(need, device=device)[:, None]
    at = (start[:, None] + j[None, :]).clamp(max=n_pages - 1)
    return torch.where(used, order[at], torch.full_like(order[at], -1)).contiguous(), n_pages


def _offsets(counts, device):
    cu = [0]
    for m in counts:
        cu.append(cu[-1] + m)
    row_b = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    row_i = torch.arange(cu[-1]) - torch.tensor(cu[:-1])[row_b]
    return torch.tensor(cu, dtype=torch.int32, device=device), row_b.to(device), row_i.to(device)


def prepare(case, seed):
    c, device = dict(case), torch.device("cuda")
    g = _gen(seed, device)
    B, H, D, P = c["batch"], c["kv_heads"], c["head_dim"], c["page"]
    lens = _lengths(c)
    s = {"case": c, "lens": torch.tensor(lens, dtype=torch.int32, device=device)}
    held = [t + m for t, m in zip(lens, _counts(c))] if c["op"] == "append" else lens
    capacity = max(max(held), 1)
    s["table"], n_pages = _paged(c, held, capacity, g, device)
    s["k_codes"], s["k_scales"] = _quantised(n_pages, c, g, device)
    s["v_codes"], s["v_scales"] = _quantised(n_pages, c, g, device)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=device)
    dt = DTYPE[c["dtype"]]
    T = s["table"].shape[1] * P
    if c["op"] == "attend":
        counts = _counts(c)
        s["cu"], s["row_b"], s["row_i"] = _offsets(counts, device)
        s["max_q"], s["scale"], s["decay"] = max(counts), 1.0 / math.sqrt(D), 0.97
        # queries that find some keys: scores spread over a few units
        s["q"] = (1.5 * torch.randn((sum(counts), c["q_heads"], D), generator=g, device=device)).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((sum(counts), c["q_heads"]), device=device)
        if c["weights"]:
            filled = torch.arange(T, device=device)[None, None, :] < s["lens"][:, None, None]
            s["weights_in"] = torch.rand((B, H, T), generator=g, device=device) * filled
            s["weights"] = torch.zeros((B, H, T), device=device)
    elif c["op"] == "append":
        counts = _counts(c)
        s["cu"], s["row_b"], s["row_i"] = _offsets(counts, device)
        shape = (sum(counts), H, D)
        for n in ("k", "v"):
            x = torch.randn(shape, generator=g, device=device)
            s[n] = (x * _channels((1, H, D), g, device)).to(dt)
        s["begin"] = (s["lens"] // P * P).to(torch.int32)
        s["new_lens"] = torch.empty_like(s["lens"])
        W = _window(c) * P
        s["k_out"] = torch.empty((B, W, H, D), dtype=dt, device=device)
        s["v_out"] = torch.empty((B, W, H, D), dtype=dt, device=device)
    else:
        filled = torch.arange(T, device=device)[None, None, :] < s["lens"][:, None, None]
        # a few tokens hold most of the weight; some tokens were never attended at all
        w = torch.rand((B, H, T), generator=g, device=device) ** 8
        w = torch.where(torch.rand((B, H, T), generator=g, device=device) < 0.05, torch.zeros_like(w), w)
        s["weights"] = torch.where(filled, w, torch.zeros_like(w))
        kept = [min(t, c["budget"]) for t in lens]
        s["new_table"], n_new = _paged(c, kept, c["budget"], g, device)
        code = TORCH_CODE[c["code"]]
        for n in ("k", "v"):
            s["new_%s_codes" % n] = torch.zeros((n_new, H, P, D), dtype=torch.uint8, device=device).view(code)
            s["new_%s_scales" % n] = torch.zeros((n_new, H), device=device)
            s["%s_out" % n] = torch.empty((B, c["budget"], H, D), dtype=dt, device=device)
        s["new_lens"] = torch.empty_like(s["lens"])
        s["new_weights"] = torch.empty((B, H, c["budget"]), device=device)
        s["kept"] = torch.empty((B, H, c["budget"]), dtype=torch.int32, device=device)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _RUN_OWN[state["case"]["op"]](state)
    return _RUN_PLAIN[state["case"]["op"]](state)


def _handles(s):
    """The cache handles and the workspace that a program keeps beside its cache."""
    import lossless_bit_level_gb300 as ibp

    c = s["case"]
    h = s["handles"] = {"ibp": ibp}
    h["cache"] = ibp.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["table"], s["lens"])
    if c["op"] == "attend":
        n = ibp.kv_attention_scratch_bytes(h["cache"], s["q"].shape[0], s["max_q"], c["q_heads"], c["weights"])
    elif c["op"] == "append":
        h["after"] = ibp.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["table"], s["new_lens"])
        n = 0
    else:
        h["new"] = ibp.KVCache(s["new_k_codes"], s["new_v_codes"], s["new_k_scales"], s["new_v_scales"],
                               s["new_table"], s["new_lens"])
        n = ibp.kv_evict_scratch_bytes(h["cache"], c["budget"])
    h["scratch"] = torch.empty(max(n, 16), dtype=torch.uint8, device=s["lens"].device)
    return h


def _own_attend(s):
    h = s.get("handles") or _handles(s)
    h["ibp"].kv_attention(h["cache"], s["q"], s["out"], s["scale"], h["scratch"], cu_q=s["cu"], max_q=s["max_q"],
                          lse=s["lse"], weights=s.get("weights"), weights_in=s.get("weights_in"),
                          decay=s["decay"], status=s["status"])
    return {"out": s["out"], "lse": s["lse"], "weights": s.get("weights")}


def _own_append(s):
    h = s.get("handles") or _handles(s)
    h["ibp"].kv_append(h["cache"], s["k"], s["v"], cu=s["cu"], new_lens=s["new_lens"], status=s["status"])
    h["ibp"].kv_read(h["after"], s["k_out"], s["v_out"], begin=s["begin"], status=s["status"])
    return {"k": s["k_out"], "v": s["v_out"], "lens": s["new_lens"]}


def _own_evict(s):
    h, c = s.get("handles") or _handles(s), s["case"]
    h["ibp"].kv_evict(h["cache"], s["weights"], c["budget"], c["recent"], h["new"], h["scratch"],
                      new_weights=s["new_weights"], kept=s["kept"], status=s["status"])
    h["ibp"].kv_read(h["new"], s["k_out"], s["v_out"], status=s["status"])
    return {"k": s["k_out"], "v": s["v_out"], "lens": s["new_lens"], "weights": s["new_weights"], "kept": s["kept"]}


_RUN_OWN = {"attend": _own_attend, "append": _own_append, "evict": _own_evict}


# the plain forms

def _as_float(code_bytes, c):
    """Whole bytes (torch.uint8) as the numbers that the codes are."""
    return code_bytes.view(TORCH_CODE[c["code"]]).float()


def _gathered(codes, scales, table, c):
    """Values [B, H, columns * page, D] of every slot that a table names."""
    ids = table.clamp(min=0).long()
    x = _as_float(codes.view(torch.uint8)[ids], c) * scales[ids][..., None, None]
    B, n, H, P, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, n * P, D)


def _plain_attend(s):
    c = s["case"]
    k = _gathered(s["k_codes"], s["k_scales"], s["table"], c)
    v = _gathered(s["v_codes"], s["v_scales"], s["table"], c)
    B, H, T, D = k.shape
    Hq, Q = c["q_heads"], s["max_q"]
    G = Hq // H
    cu, lens = s["cu"].long(), s["lens"].long()
    counts = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=k.device)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().reshape(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, D)
    x = (q @ k.transpose(2, 3)) * s["scale"]
    limit = (lens - counts)[:, None] + i[None, :] + 1
    limit = torch.where(i[None, :] < counts[:, None], limit, torch.zeros_like(limit))
    seen = torch.arange(T, device=k.device)[None, None, :] < limit[:, :, None]
    seen = seen[:, None, None].expand(B, 1, G, Q, T).reshape(B, 1, G * Q, T)
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(x - top)
    del x
    total = e.sum(-1, keepdim=True)
    inverse = torch.where(total > 0, 1.0 / total, torch.zeros_like(total))
    o = (e @ v) * inverse
    lse = top + torch.log(total)
    b, r = s["row_b"], s["row_i"]
    out = o.reshape(B, H, G, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)[b, r].to(s["q"].dtype)
    lse = lse.reshape(B, H, G, Q).permute(0, 3, 1, 2).reshape(B, Q, Hq)[b, r]
    weights = None
    if c["weights"]:
        filled = torch.arange(T, device=k.device)[None, None, :] < lens[:, None, None]
        weights = s["decay"] * s["weights_in"] + (e * inverse).sum(2)
        weights = torch.where(filled, weights, torch.zeros_like(weights))
    return {"out": out, "lse": lse, "weights": weights}


def _scale_of(largest, c):
    scale = (largest / QMAX[c["code"]]).clamp(SMALLEST, LARGEST)
    return torch.where(largest > 0, scale, torch.zeros_like(scale))


def _coded(x, c):
    """The numbers that x, already divided by its scale, is held as."""
    if c["code"] == "int8":
        return x.round().clamp(-127.0, 127.0)
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()


def _inverse_of(scale):
    return torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))


def _plain_append(s):
    c = s["case"]
    P, H, D, B = c["page"], c["kv_heads"], c["head_dim"], c["batch"]
    cu, lens = s["cu"].long(), s["lens"].long()
    counts = cu[1:] - cu[:-1]
    W = s["k_out"].shape[1]
    at = s["begin"].long()[:, None] + torch.arange(W, device=lens.device)[None, :]
    old, new = at < lens[:, None], at < (lens + counts)[:, None]
    new = new & ~old
    rows = (cu[:-1, None] + at - lens[:, None]).clamp(0, s["k"].shape[0] - 1)
    pages = (at[:, ::P] // P).clamp(max=s["table"].shape[1] - 1)
    ids = torch.gather(s["table"], 1, pages).clamp(min=0).long()
    partly = (old[:, ::P])[:, :, None]
    got = {}
    for n in ("k", "v"):
        x = torch.where(new[:, :, None, None], s[n][rows].float(), torch.zeros((), device=lens.device))
        x = x.reshape(B, W // P, P, H, D)
        before = torch.where(partly, s[n + "_scales"][ids], torch.zeros((), device=lens.device))
        scale = torch.maximum(before, _scale_of(x.abs().amax((2, 4)), c))
        inverse = _inverse_of(scale)
        there = _as_float(s[n + "_codes"].view(torch.uint8)[ids], c).permute(0, 1, 3, 2, 4)
        ratio = before * inverse
        ratio = torch.where(scale > before, before / scale, torch.ones_like(ratio))
        there = torch.where((scale > before)[:, :, None, :, None], _coded(there * ratio[:, :, None, :, None], c), there)
        code = torch.where(new.reshape(B, W // P, P, 1, 1), _coded(x * inverse[:, :, None, :, None], c), there)
        value = (code * scale[:, :, None, :, None]).reshape(B, W, H, D)
        value = torch.where((old | new)[:, :, None, None], value, torch.zeros_like(value))
        got[n] = value.to(s[n].dtype)
    return {"k": got["k"], "v": got["v"], "lens": (lens + counts).to(torch.int32)}


def _plain_evict(s):
    c = s["case"]
    P, D, budget, recent = c["page"], c["head_dim"], c["budget"], c["recent"]
    B, H, T = s["weights"].shape
    lens = s["lens"].long()
    t = torch.arange(T, device=lens.device)[None, None, :]
    n = lens[:, None, None]
    rank = torch.where(t >= n - recent, torch.full_like(s["weights"], math.inf), s["weights"])
    rank = torch.where(t >= n, torch.full_like(rank, -math.inf), rank)
    order = torch.sort(rank, dim=2, descending=True, stable=True)[1][:, :, :budget]
    if order.shape[2] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[2]), value=T)
    slot = torch.arange(budget, device=lens.device)[None, None, :]
    order = torch.where(slot < n.clamp(max=budget), order, torch.full_like(order, T))
    kept = torch.sort(order, dim=2)[0]
    there = kept < T
    at = kept.clamp(max=T - 1)
    weights = torch.where(there, torch.gather(s["weights"], 2, at), torch.zeros((), device=lens.device))
    ids = torch.gather(s["table"].long()[:, None, :].expand(B, H, -1), 2, at // P).clamp(min=0)
    heads = torch.arange(H, device=lens.device)[None, :, None].expand_as(ids)
    full = _pages(budget, P) * P
    got = {}
    for name in ("k", "v"):
        code = _as_float(s[name + "_codes"].view(torch.uint8)[ids, heads, at % P], c)
        x = code * s[name + "_scales"][ids, heads][..., None]
        x = torch.where(there[..., None], x, torch.zeros_like(x))
        x = torch.nn.functional.pad(x, (0, 0, 0, full - budget)).reshape(B, H, full // P, P, D)
        scale = _scale_of(x.abs().amax((3, 4)), c)
        x = _coded(x * _inverse_of(scale)[..., None, None], c) * scale[..., None, None]
        x = x.reshape(B, H, full, D)[:, :, :budget].transpose(1, 2).contiguous()
        got[name] = x.to(DTYPE[c["dtype"]])
    kept = torch.where(there, kept, torch.full_like(kept, -1)).to(torch.int32)
    return {"k": got["k"], "v": got["v"], "lens": lens.clamp(max=budget).to(torch.int32), "weights": weights, "kept": kept}


_RUN_PLAIN = {"attend": _plain_attend, "append": _plain_append, "evict": _plain_evict}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "evict": _exact_evict}[case["op"]](s, dict(case))


def _tokens(s, name, b, length, c, heads=slice(None)):
    """Values of the first `length` tokens of sequence b in 64 bits: [heads, length, D]."""
    ids = s["table"][b, :_pages(length, c["page"])].long()
    raw = s[name + "_codes"].view(torch.uint8)[ids][:, heads].view(TORCH_CODE[c["code"]])
    x = raw.float().double() * s[name + "_scales"][ids][:, heads].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, c["head_dim"])[:, :length]


def _exact_attend(s, c):
    lens, counts = _lengths(c), _counts(c)
    H, Hq = c["kv_heads"], c["q_heads"]
    G, first = Hq // H, 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    weights = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda") if c["weights"] else None
    for b, (t, m) in enumerate(zip(lens, counts)):
        if t:
            for h in range(H):
                k = _tokens(s, "k", b, t, c, slice(h, h + 1))[0]
                v = _tokens(s, "v", b, t, c, slice(h, h + 1))[0]
                dead = torch.arange(t, device="cuda")[None, :] > torch.arange(t - m, t, device="cuda")[:, None]
                for a in range(G):
                    x = s["q"][first:first + m, h * G + a].double() @ k.T / math.sqrt(c["head_dim"])
                    x.masked_fill_(dead, -math.inf)
                    z = torch.logsumexp(x, 1)
                    p = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
                    out[first:first + m, h * G + a] = p @ v
                    lse[first:first + m, h * G + a] = z
                    if weights is not None:
                        weights[b, h, :t] += p.sum(0)
        first += m
    if weights is not None:
        weights += s["decay"] * s["weights_in"].double()
    return {"out": out, "lse": lse, "weights": weights}


def _exact_page(x, c, before, old):
    """One page's values [tokens, D]: `old` codes held at the scale `before`, then the values x."""
    top = QMAX[c["code"]]
    finest = float(x.abs().max()) if x.numel() else 0.0
    scale = min(max(finest / top, SMALLEST), LARGEST) if finest > 0 else 0.0
    scale = max(scale, before)

    def held(y):
        y = y.clamp(-top, top)
        if c["code"] == "int8":
            return y.round()
        return _e4m3(y)

    new = held(x / scale) * scale if scale > 0 else torch.zeros_like(x)
    return torch.cat([held(old * (before / scale)) * scale if scale > before else old * before, new])


def _e4m3(y):
    """The nearest number with a sign, 3 bits behind the point and exponents from -6 up; ties to even."""
    exponent = torch.frexp(y)[1].clamp(min=-5) - 4
    unit = torch.ldexp(torch.ones_like(y), exponent)
    return torch.round(y / unit) * unit


def _exact_append(s, c):
    lens, counts, P = _lengths(c), _counts(c), c["page"]
    H, cu, got = c["kv_heads"], s["cu"].tolist(), {}
    for n in ("k", "v"):
        value = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
        for b, (t, m) in enumerate(zip(lens, counts)):
            rows, off = s[n][cu[b]:cu[b + 1]].double(), t % P
            first = min(m, P - off) if off else 0  # rows that join a partly filled page
            if off:
                page = int(s["table"][b, t // P])
                for h in range(H):
                    raw = s[n + "_codes"].view(torch.uint8)[page, h, :off]
                    old = raw.view(TORCH_CODE[c["code"]]).float().double()
                    before = float(s[n + "_scales"][page, h])
                    value[b, :off + first, h] = _exact_page(rows[:first, h], c, before, old)
            if m > first:
                start = P if off else 0
                value[b, start:start + m - first] = _exact_pages(rows[first:], c)
        got[n] = value
    return {"k": got["k"], "v": got["v"], "lens": None}


def _exact_pages(x, c):
    """Rows [tokens, H, D] quantised into pages that start empty."""
    P, top, (m, H, D) = c["page"], QMAX[c["code"]], x.shape
    y = torch.zeros((_pages(m, P) * P, H, D), dtype=torch.float64, device=x.device)
    y[:m] = x
    y = y.reshape(-1, P, H, D)
    largest = y.abs().amax((1, 3), keepdim=True)
    scale = torch.where(largest > 0, (largest / top).clamp(SMALLEST, LARGEST), torch.zeros_like(largest))
    y = (y / torch.where(scale > 0, scale, torch.ones_like(scale))).clamp(-top, top)
    y = (y.round() if c["code"] == "int8" else _e4m3(y)) * scale
    return y.reshape(-1, H, D)[:m]


def _exact_evict(s, c):
    lens, H, budget, recent = _lengths(c), c["kv_heads"], c["budget"], c["recent"]
    got = {n: torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for n in ("k", "v")}
    weights = torch.zeros(s["new_weights"].shape, dtype=torch.float64, device="cuda")
    for b, t in enumerate(lens):
        held = {n: _tokens(s, n, b, t, c) for n in ("k", "v")}
        for h in range(H):
            w = s["weights"][b, h, :t].double()
            if t > budget:
                early = torch.argsort(-w[:t - recent], stable=True)[:budget - recent]
                keep = torch.cat([early.sort()[0], torch.arange(t - recent, t, device="cuda")])
            else:
                keep = torch.arange(t, device="cuda")
            weights[b, h, :keep.numel()] = w[keep]
            for n in ("k", "v"):
                got[n][b, :keep.numel(), h] = _exact_pages(held[n][h, keep][:, None], c)[:, 0]
    return {"k": got["k"], "v": got["v"], "lens": None, "weights": weights, "kept": None}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(k)) for k in range(6)]:
        print(case, work(case))
