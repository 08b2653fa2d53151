"""What the serving operators around the 8-bit key/value cache are measured on.

The operators: rows of keys and values put into the paged cache with the position rotation
applied on the way, to the queries as well (rotate); attention of a batch whose sequences
share long beginnings, each beginning gone over once for all of them (share); and attention
over the pages that a cheap score selects for each sequence and head, with the pages' bounds
that the score goes by kept up to date (select).

The cache is that of perf/operators.py: codes [pages, heads, page_tokens, head_dim] (int8 or
float8 e4m3), scales [pages, heads], a page table [batch, columns] and lengths [batch]; a
value is code * scale. A page whose largest finite magnitude is a has the scale a * (1/qmax)
held in [2^-100, 2^120] (0 where a is 0); rows appended to a page that is partly filled raise
its scale where they need to, and the codes that are there are rescaled.

Rotation: table[p, i] holds the cosine and sine of pair i at position p, pair i of a head's
first `dim` elements is (i, i + dim/2), or (2i, 2i + 1) where interleaved, and goes by the
position on its axis. (x, y) becomes (x c - y s, y c + x s), each product and sum rounded to
32 bits; keys are quantised from that, queries rounded once to their type.

Bounds of a page: for each head and element the least and the largest code of the page's
tokens, for e4m3 in units of 448/127 of a code, rounded outwards: whole numbers in
[-127, 127]. The score of a page for a query row whose largest magnitude is in [2^e, 2^(e+1)):
with n_d = q_d * 2^(6-e) rounded to nearest even and held in [-127, 127], the whole number
s = sum_d max(n_d * least_d, n_d * largest_d), times 2^(e-6) and then the page's key scale; of
a sequence's rows and the query heads of one key/value head the largest counts. Selected are
the first page, the last ones (as many as the query rows stand in, one at least), and of the
others those of the highest scores, the lowest page first where scores are equal.
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
        # one new token for each of a batch of conversations
        dict(name="rotate tokens", op="rotate", batch=64, q_heads=32, kv_heads=8, head_dim=128, page=64,
             code="int8", dtype="bf16", longest=4_000, shortest=1, rows=1, even=True, dim=128, axes=1,
             interleaved=False),
        # the whole prompts of one decoder layer as this repository stores it (8 x 4096 tokens,
        # 32 heads of 128, no shared heads)
        dict(name="rotate layer", op="rotate", batch=8, q_heads=32, kv_heads=32, head_dim=128, page=64,
             code="int8", dtype="bf16", longest=0, shortest=0, rows=4_096, even=True, dim=128, axes=1,
             interleaved=False),
        # prompts with frames of a video among the text: positions on three axes
        dict(name="rotate frames", op="rotate", batch=5, q_heads=28, kv_heads=4, head_dim=128, page=32,
             code="e4m3", dtype="fp16", longest=901, shortest=0, rows=2_222, even=False, dim=128, axes=3,
             interleaved=False),
        # ragged pieces of prompts in 32 bits behind pages that are partly filled, half of each
        # head rotated in neighbouring pairs
        dict(name="rotate pieces", op="rotate", batch=21, q_heads=8, kv_heads=8, head_dim=64, page=16,
             code="e4m3", dtype="fp32", longest=1_501, shortest=3, rows=333, even=False, dim=32, axes=1,
             interleaved=True),
        # a few short conversations behind one instruction: a call whose latency is what counts
        dict(name="share few", op="share", batch=4, groups=1, q_heads=32, kv_heads=8, head_dim=128, page=16,
             code="int8", dtype="bf16", prefix=777, prefix_low=777, longest=100, shortest=1, queries=1,
             even=True),
        # conversations of a service behind one long instruction
        dict(name="share chats", op="share", batch=32, groups=1, q_heads=32, kv_heads=8, head_dim=128, page=64,
             code="int8", dtype="bf16", prefix=8_192, prefix_low=8_192, longest=900, shortest=1, queries=1,
             even=True),
        # several answers to each of two long documents, no two equally long
        dict(name="share documents", op="share", batch=16, groups=2, q_heads=32, kv_heads=4, head_dim=128,
             page=64, code="e4m3", dtype="bf16", prefix=60_001, prefix_low=33_333, longest=700, shortest=0,
             queries=1, even=True),
        # a ragged batch behind three prompts that checks a few proposed tokens a sequence
        dict(name="share verify", op="share", batch=40, groups=3, q_heads=16, kv_heads=4, head_dim=64, page=32,
             code="int8", dtype="fp16", prefix=4_001, prefix_low=0, longest=1_003, shortest=0, queries=7,
             even=False),
        # one conversation, one query token: a call whose latency is what counts
        dict(name="select one", op="select", batch=1, q_heads=32, kv_heads=8, head_dim=128, page=16,
             code="int8", dtype="bf16", longest=7_777, shortest=7_777, queries=1, even=True, pages=64,
             bounds="new"),
        # one decoder layer of this repository's size after its prompts: every page's bounds
        dict(name="select layer", op="select", batch=8, q_heads=32, kv_heads=32, head_dim=128, page=64,
             code="int8", dtype="bf16", longest=4_096, shortest=4_096, queries=1, even=True, pages=16,
             bounds="all"),
        # long documents, a token each
        dict(name="select long", op="select", batch=16, q_heads=32, kv_heads=8, head_dim=128, page=32,
             code="e4m3", dtype="bf16", longest=60_001, shortest=35_000, queries=1, even=True, pages=64,
             bounds="new"),
        # a ragged batch (an empty sequence among it) that checks a few proposed tokens a sequence
        dict(name="select verify", op="select", batch=48, q_heads=16, kv_heads=4, head_dim=64, page=32,
             code="int8", dtype="fp16", longest=7_003, shortest=0, queries=7, even=False, pages=24,
             bounds="new"),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        # no more than the largest listed cases: bytes moved, operations, and elements held
        held = c["kv_heads"] * c["head_dim"] * sum(_lengths(c))
        if c["op"] == "rotate":
            spread = c["batch"] * c["kv_heads"] * c["head_dim"] * (c["longest"] + c["rows"])
            if w["bytes"] <= 1.8e9 and spread <= 1.4e8:
                return c
        elif c["op"] == "share":
            spread = c["batch"] * c["kv_heads"] * c["head_dim"] * (c["prefix"] + c["longest"])
            scores = c["batch"] * c["q_heads"] * c["queries"] * (c["prefix"] + c["longest"])
            if spread <= 5.0e8 and scores <= 3.2e7 and w["flops"] <= 1.6e10:
                return c
        else:
            chosen = c["batch"] * c["kv_heads"] * c["head_dim"] * min(c["pages"] * c["page"], c["longest"])
            built = held if c["bounds"] == "all" else 0
            if held <= 8.0e8 and chosen <= 5.4e7 and built <= 1.4e8 and w["flops"] <= 5.0e9:
                return c


def _draw(rng):
    op = rng.choice(["rotate", "share", "select"])
    batch = _log(rng, 1, 64)
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    c = dict(op=op, batch=batch, kv_heads=kv_heads, head_dim=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128]), code=rng.choice(["int8", "int8", "e4m3"]),
             q_heads=kv_heads * rng.choice([1, 2, 4, 8, 5]))
    if op == "rotate":
        longest = rng.choice([0, _log(rng, 1, 8_000)])
        c.update(dtype=rng.choice(["bf16", "fp16", "fp32"]), longest=longest,
                 shortest=min(longest, rng.choice([0, 1, longest // 3, longest])),
                 rows=rng.choice([1, _log(rng, 1, 4_096)]), even=rng.random() < 0.5,
                 dim=rng.choice([c["head_dim"], c["head_dim"], c["head_dim"] // 2, 16, 48]),
                 axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4)
        return c
    queries = rng.choice([1, 1, 1, _log(rng, 1, 8)])
    if op == "share":
        prefix, longest = _log(rng, 1, 60_000), _log(rng, 1, 4_000)
        c.update(dtype=rng.choice(["bf16", "fp16"]), groups=min(batch, rng.choice([1, 1, 2, 3, 5])),
                 prefix=prefix, prefix_low=rng.choice([0, prefix // 3, prefix]), longest=longest,
                 shortest=min(longest, rng.choice([0, 1, longest])), queries=queries,
                 even=rng.random() < 0.5)
        return c
    longest = _log(rng, 1, 120_000)
    least = -(-(queries - 1) // c["page"]) + 2
    c.update(dtype=rng.choice(["bf16", "fp16"]), longest=longest,
             shortest=min(longest, rng.choice([0, 1, longest // 3, longest])), queries=queries,
             even=rng.random() < 0.5, pages=max(least, _log(rng, 2, 256)),
             bounds=rng.choice(["new", "new", "all"]))
    return c


# ------------------------------------------- sizes that follow from a case alone

def _spread(low, high, n):
    """n whole numbers from high down to low, spread as a low-discrepancy sequence."""
    if n == 1:
        return [high]
    return [high, low] + [low + int((high - low + 1) * ((0.6180339887 * i) % 1.0)) for i in range(1, n - 1)]


def _group_of(c):
    return [b * c["groups"] // c["batch"] for b in range(c["batch"])]


def _prefixes(c):
    return _spread(c["prefix_low"], c["prefix"], c["groups"])


def _lengths(c):
    """Tokens that each sequence holds before the call."""
    mine = _spread(c["shortest"], c["longest"], c["batch"])
    if c["op"] != "share":
        return mine
    prefix = _prefixes(c)
    return [prefix[g] + t for g, t in zip(_group_of(c), mine)]


def _counts(c):
    """New rows (rotate) or query rows (share, select) of each sequence."""
    most = c["rows"] if c["op"] == "rotate" else c["queries"]
    return [most] * c["batch"] if c["even"] else _spread(1, most, c["batch"])


def _pages(n, page):
    return -(-n // page)


def _window(c):
    """Pages that the new rows of one sequence touch, at most."""
    P = c["page"]
    return max(_pages(t + m, P) - t // P for t, m in zip(_lengths(c), _counts(c)))


def _begins(c):
    """First token whose page's bounds a call brings up to date."""
    if c["bounds"] == "all":
        return [0] * c["batch"]
    return [max(t - m, 0) for t, m in zip(_lengths(c), _counts(c))]


def _axis(c):
    """The axis of each pair: a quarter of them time, the rest height and width in halves."""
    n, axes = c["dim"] // 2, c["axes"]
    first = n if axes == 1 else n // 4
    return [0] * first + [1 + (i * (axes - 1)) // (n - first) for i in range(n - first)]


def work(case):
    c = case
    H, D, P, Hq, es = c["kv_heads"], c["head_dim"], c["page"], c["q_heads"], SIZE[c["dtype"]]
    lens, counts = _lengths(c), _counts(c)
    n = sum(counts)
    if c["op"] == "rotate":
        window = _window(c) * P * c["batch"]
        # rows read, their codes written, the touched pages' values written, queries turned
        nbytes = 2 * H * D * (n * es + n + window * es) + 2 * n * Hq * D * es
        return {"bytes": nbytes, "flops": 6 * 2 * H * D * n + 3 * c["dim"] * (H + Hq) * n}
    pairs = sum(sum(max(0, t - m + i + 1) for i in range(m)) for t, m in zip(lens, counts))
    nbytes = 2 * n * Hq * D * es + 4 * n * Hq
    if c["op"] == "share":
        prefix, size = _prefixes(c), [_group_of(c).count(g) for g in range(c["groups"])]
        held = sum(lens) - sum(p * (s - 1) for p, s in zip(prefix, size) if s)
        return {"bytes": nbytes + 2 * held * H * D + 8 * _pages(held, P) * H, "flops": 4 * Hq * D * pairs}
    tokens = sum(min(t, c["pages"] * P) for t in lens)
    pages = sum(_pages(t, P) for t in lens)
    fresh = sum(t - a // P * P for t, a in zip(lens, _begins(c)))
    seen = sum(min(t, c["pages"] * P) * m for t, m in zip(lens, counts))
    # new bounds from codes; bounds and key scales of all pages; the selected pages' codes
    nbytes += fresh * H * D + 2 * _pages(fresh, P) * H * D + pages * H * (2 * D + 4) + 2 * tokens * H * D
    score = sum(_pages(t, P) * m for t, m in zip(lens, counts)) * Hq * 4 * D
    return {"bytes": nbytes + 4 * c["batch"] * H * c["pages"], "flops": 4 * Hq * D * seen + score + 2 * fresh * H * D}


# ---------------------------------------------------------------- inputs

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
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
    # the tokens of a page are alike, so that some pages matter more than others
    x += 1.5 * torch.randn((n_pages, H, 1, D), generator=g, device=device)
    s = x.abs().amax((2, 3)) * (1.0 / QMAX[c["code"]])
    x /= s[:, :, None, None]
    if c["code"] == "int8":
        return x.round_().clamp_(-127.0, 127.0).to(torch.int8), s
    return x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _table(first, whole, rest, n_pages, cols, g, device):
    """A page table in random page order: sequence b's columns below whole[b] are pages
    first[b][0] .., the rest[b] columns after them pages first[b][1] ..."""
    order = torch.randperm(n_pages, generator=g, device=device).to(torch.int32)
    a, o = (torch.tensor([f[k] for f in first], device=device)[:, None] for k in range(2))
    w, r = (torch.tensor(x, device=device)[:, None] for x in (whole, rest))
    j = torch.arange(max(cols, 1), device=device)[None, :]
    at = torch.where(j < w, a + j, o + j - w).clamp(min=0, max=n_pages - 1)
    return torch.where(j < w + r, order[at], torch.full_like(order[at], -1)).contiguous()


def _offsets(counts, device):
    cu = [0]
    for m in counts:
        cu.append(cu[-1] + m)
    row_b = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    row_i = torch.arange(cu[-1]) - torch.tensor(cu[:-1])[row_b]
    return torch.tensor(cu, dtype=torch.int32, device=device), row_b.to(device), row_i.to(device)


def _int32(x, device):
    return torch.tensor(x, dtype=torch.int32, device=device)


def prepare(case, seed):
    c, device = dict(case), torch.device("cuda")
    g = _gen(seed, device)
    B, H, D, P = c["batch"], c["kv_heads"], c["head_dim"], c["page"]
    lens, counts = _lengths(c), _counts(c)
    s = {"case": c, "lens": _int32(lens, device)}
    held = [t + m for t, m in zip(lens, counts)] if c["op"] == "rotate" else lens
    need, whole = [_pages(t, P) for t in held], [0] * B
    starts, at = [], 0
    if c["op"] == "share":
        group, prefix = _group_of(c), _prefixes(c)
        whole = [prefix[k] // P for k in group]
        shared = []
        for p in prefix:
            shared.append(at)
            at += p // P
    for b in range(B):
        starts.append((shared[group[b]] if c["op"] == "share" else 0, at))
        at += need[b] - whole[b]
    n_pages = at + 3
    s["table"] = _table(starts, whole, [n - w for n, w in zip(need, whole)], n_pages, max(need), g, device)
    s["k_codes"], s["k_scales"] = _quantised(n_pages, c, g, device)
    s["v_codes"], s["v_scales"] = _quantised(n_pages, c, g, device)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=device)
    s["cu"], s["row_b"], s["row_i"] = _offsets(counts, device)
    dt, n = DTYPE[c["dtype"]], sum(counts)
    # queries that find some keys: scores spread over a few units
    s["q"] = (1.5 * torch.randn((n, c["q_heads"], D), generator=g, device=device)).to(dt)
    if c["op"] == "rotate":
        _prepare_rotate(s, c, g, device)
        return s
    s["max_q"], s["scale"] = max(counts), 1.0 / math.sqrt(D)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((n, c["q_heads"]), device=device)
    if c["op"] == "share":
        first = [group.index(k) if k in group else B for k in range(c["groups"])] + [B]
        s["groups"], s["prefix"] = _int32(first, device), _int32(prefix, device)
        s["group_rows"] = max(sum(m for m, k in zip(counts, group) if k == x) for x in range(c["groups"]))
    else:
        s["begin"] = _int32(_begins(c), device)
        s["bounds"] = _old_bounds(s, c)
        s["columns"] = torch.empty((B, H, c["pages"]), dtype=torch.int32, device=device)
    return s


def _prepare_rotate(s, c, g, device):
    B, H, D, P = c["batch"], c["kv_heads"], c["head_dim"], c["page"]
    lens, counts, dt = _lengths(c), _counts(c), DTYPE[c["dtype"]]
    n = sum(counts)
    for name in ("k", "v"):
        x = torch.randn((n, H, D), generator=g, device=device)
        s[name] = (x * _channels((1, H, D), g, device)).to(dt)
    s["q_out"] = torch.empty_like(s["q"])
    far = max(t + m for t, m in zip(lens, counts))
    if c["axes"] == 1:
        s["positions"] = None  # a token's place in its sequence
    else:  # frames of 24 x 36 patches among the text
        t = s["lens"][s["row_b"]].long() + s["row_i"]
        axes = [t] + [t // (864 if k == 0 else 36) % (24 if k == 0 else 36) + t // 864 for k in range(c["axes"] - 1)]
        s["positions"] = torch.stack(axes, 1).to(torch.int32).contiguous()
        far += 36
    pairs = c["dim"] // 2
    inverse = 10_000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=device) / pairs)
    angle = torch.arange(far, dtype=torch.float64, device=device)[:, None] * inverse[None, :]
    s["turns"] = torch.stack([angle.cos(), angle.sin()], 2).float().contiguous()
    s["axis"] = _axis(c)
    s["begin"] = (s["lens"] // P * P).to(torch.int32)
    s["new_lens"] = torch.empty_like(s["lens"])
    W = _window(c) * P
    s["k_out"] = torch.empty((B, W, H, D), dtype=dt, device=device)
    s["v_out"] = torch.empty((B, W, H, D), dtype=dt, device=device)


def _old_bounds(s, c):
    """Bounds as earlier calls left them; those of pages that a call brings up to date are zeros."""
    B, P = c["batch"], c["page"]
    out = torch.zeros((s["k_codes"].shape[0], c["kv_heads"], 2, c["head_dim"]), dtype=torch.int8,
                      device=s["lens"].device)
    step = max(1, (1 << 27) // (c["kv_heads"] * P * c["head_dim"]))
    for a in range(0, out.shape[0], step):
        x = _as_float(s["k_codes"].view(torch.uint8)[a:a + step], c)
        out[a:a + step, :, 0], out[a:a + step, :, 1] = _outwards(x.amin(2), x.amax(2), c)
    j = torch.arange(s["table"].shape[1], device=out.device)[None, :]
    stale = (j >= s["begin"][:, None] // P) & (s["table"] >= 0)
    out[s["table"][stale].long()] = 0
    used = torch.zeros(out.shape[0], dtype=torch.bool, device=out.device)
    used[s["table"][s["table"] >= 0].long()] = True
    out[~used] = 0
    return out


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
    n = 0
    if c["op"] == "rotate":
        h["after"] = ibp.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["table"], s["new_lens"])
        h["rotation"] = ibp.KVRotation(s["turns"], axis=s["axis"], interleaved=c["interleaved"])
    elif c["op"] == "share":
        n = ibp.kv_attention_shared_scratch_bytes(h["cache"], s["q"].shape[0], s["max_q"], c["q_heads"],
                                                  c["groups"], s["group_rows"])
    else:
        n = max(ibp.kv_select_scratch_bytes(h["cache"]),
                ibp.kv_attention_selected_scratch_bytes(h["cache"], s["q"].shape[0], s["max_q"], c["q_heads"],
                                                        c["pages"]))
    h["scratch"] = torch.empty(max(n, 16), dtype=torch.uint8, device=s["lens"].device)
    return h


def _own_rotate(s):
    h = s.get("handles") or _handles(s)
    h["ibp"].kv_append_rotated(h["cache"], s["k"], s["v"], h["rotation"], positions=s["positions"], q=s["q"],
                               q_out=s["q_out"], cu=s["cu"], new_lens=s["new_lens"], status=s["status"])
    h["ibp"].kv_read(h["after"], s["k_out"], s["v_out"], begin=s["begin"], status=s["status"])
    return {"k": s["k_out"], "v": s["v_out"], "q": s["q_out"], "lens": s["new_lens"]}


def _own_share(s):
    h = s.get("handles") or _handles(s)
    h["ibp"].kv_attention_shared(h["cache"], s["q"], s["out"], s["scale"], h["scratch"], s["groups"], s["prefix"],
                                 s["group_rows"], cu_q=s["cu"], max_q=s["max_q"], lse=s["lse"], status=s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_select(s):
    h, c = s.get("handles") or _handles(s), s["case"]
    h["ibp"].kv_bounds(h["cache"], s["bounds"], begin=s["begin"], status=s["status"])
    h["ibp"].kv_select(h["cache"], s["bounds"], s["q"], s["columns"], h["scratch"], cu_q=s["cu"], max_q=s["max_q"],
                       status=s["status"])
    h["ibp"].kv_attention_selected(h["cache"], s["columns"], s["q"], s["out"], s["scale"], h["scratch"],
                                   cu_q=s["cu"], max_q=s["max_q"], lse=s["lse"], status=s["status"])
    return {"bounds": s["bounds"], "columns": s["columns"], "out": s["out"], "lse": s["lse"]}


_RUN_OWN = {"rotate": _own_rotate, "share": _own_share, "select": _own_select}


# the plain forms

def _as_float(code_bytes, c):
    """Whole bytes (torch.uint8) as the numbers that the codes are."""
    return code_bytes.view(TORCH_CODE[c["code"]]).float()


def _turned(x, s, c):
    """Rows [n, heads, D] in 32 bits, each pair turned by its position's angle."""
    dim = c["dim"]
    where = s["lens"][s["row_b"]].long() + s["row_i"]
    where = where[:, None] if s["positions"] is None else s["positions"].long()
    pair = torch.arange(dim // 2, device=x.device)
    turn = s["turns"][where[:, torch.tensor(s["axis"], device=x.device)], pair[None, :]]
    cos, sin = turn[:, None, :, 0], turn[:, None, :, 1]
    a, b = (pair * 2, pair * 2 + 1) if c["interleaved"] else (pair, pair + dim // 2)
    u, v = x[..., a], x[..., b]
    y = x.clone()
    y[..., a] = u * cos - v * sin
    y[..., b] = v * cos + u * sin
    return y


def _scale_of(largest, c):
    scale = (largest * (1.0 / QMAX[c["code"]])).clamp(SMALLEST, LARGEST)
    return torch.where(largest > 0, scale, torch.zeros_like(scale))


def _coded(x, c):
    """The numbers that x, already divided by its scale, is held as."""
    if c["code"] == "int8":
        return x.round().clamp(-127.0, 127.0)
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()


def _plain_rotate(s):
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
    nothing = torch.zeros((), device=lens.device)
    got = {}
    for n in ("k", "v"):
        x = s[n].float()
        if n == "k":
            x = _turned(x, s, c)
        x = torch.where(new[:, :, None, None], x[rows], nothing).reshape(B, W // P, P, H, D)
        before = torch.where(partly, s[n + "_scales"][ids], nothing)
        scale = torch.maximum(before, _scale_of(x.abs().amax((2, 4)), c))
        inverse = torch.where(scale > 0, 1.0 / scale, nothing)
        there = _as_float(s[n + "_codes"].view(torch.uint8)[ids], c).permute(0, 1, 3, 2, 4)
        grown = scale > before
        ratio = torch.where(grown, before / scale, nothing)
        there = torch.where(grown[:, :, None, :, None], _coded(there * ratio[:, :, None, :, None], c), there)
        code = torch.where(new.reshape(B, W // P, P, 1, 1), _coded(x * inverse[:, :, None, :, None], c), there)
        value = (code * scale[:, :, None, :, None]).reshape(B, W, H, D)
        value = torch.where((old | new)[:, :, None, None], value, nothing)
        got[n] = value.to(s[n].dtype)
    got["q"] = _turned(s["q"].float(), s, c).to(s["q"].dtype)
    return {"k": got["k"], "v": got["v"], "q": got["q"], "lens": (lens + counts).to(torch.int32)}


def _rows_apart(s, c):
    """Query rows as [B, H, G * Q, D] in 32 bits, and the position of row i of each sequence."""
    cu, B, H, Q = s["cu"].long(), c["batch"], c["kv_heads"], s["max_q"]
    G, D = c["q_heads"] // H, c["head_dim"]
    counts = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=cu.device)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().reshape(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, D)
    place = (s["lens"].long() - counts)[:, None] + i[None, :]
    return q, torch.where(i[None, :] < counts[:, None], place, torch.full_like(place, -1))


def _attend(q, k, v, place, t, s, c):
    """softmax(scale * q k) v over the tokens t [B, H or 1, T] that are there (>= 0) and not past a row."""
    B, H, R, D = q.shape
    Q, Hq = s["max_q"], c["q_heads"]
    G = Hq // H
    x = (q @ k.transpose(2, 3)) * s["scale"]
    limit = place[:, None, None, :, None].expand(B, 1, G, Q, 1).reshape(B, 1, R, 1)
    seen = (t[:, :, None, :] >= 0) & (t[:, :, None, :] <= limit)
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(x - top)
    del x
    total = e.sum(-1, keepdim=True)
    o = (e @ v) * torch.where(total > 0, 1.0 / total, torch.zeros_like(total))
    lse = top + torch.log(total)
    b, r = s["row_b"], s["row_i"]
    out = o.reshape(B, H, G, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)[b, r].to(s["q"].dtype)
    return out, lse.reshape(B, H, G, Q).permute(0, 3, 1, 2).reshape(B, Q, Hq)[b, r]


def _plain_share(s):
    c = s["case"]
    ids = s["table"].clamp(min=0).long()
    B, n, P = ids.shape[0], ids.shape[1], c["page"]

    def values(name):
        x = _as_float(s[name + "_codes"].view(torch.uint8)[ids], c) * s[name + "_scales"][ids][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, c["kv_heads"], n * P, c["head_dim"])

    t = torch.arange(n * P, device=ids.device)
    t = torch.where(t[None, :] < s["lens"].long()[:, None], t[None, :], torch.full_like(t, -1)[None, :])
    q, place = _rows_apart(s, c)
    out, lse = _attend(q, values("k"), values("v"), place, t[:, None], s, c)
    return {"out": out, "lse": lse}


def _outwards(least, most, c):
    """Least and largest codes as whole numbers."""
    if c["code"] == "int8":
        return least.to(torch.int8), most.to(torch.int8)
    unit = torch.full_like(least, 448.0)  # (a tensor: a division by a number may be a product with its inverse)
    return torch.floor(least * 127.0 / unit).to(torch.int8), torch.ceil(most * 127.0 / unit).to(torch.int8)


def _plain_bounds(s, c):
    P, lens = c["page"], s["lens"].long()
    W = max(max(_pages(t, P) - a // P for t, a in zip(_lengths(c), _begins(c))), 1)
    col = (s["begin"].long() // P)[:, None] + torch.arange(W, device=lens.device)[None, :]
    here = col * P < lens[:, None]
    ids = torch.gather(s["table"].long(), 1, col.clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    x = _as_float(s["k_codes"].view(torch.uint8)[ids], c)  # [B, W, H, P, D]
    t = col[:, :, None] * P + torch.arange(P, device=lens.device)
    there = (t < lens[:, None, None])[:, :, None, :, None]
    least = torch.where(there, x, torch.full_like(x, math.inf)).amin(3)
    most = torch.where(there, x, torch.full_like(x, -math.inf)).amax(3)
    least, most = (torch.where(here[:, :, None, None], y, torch.zeros_like(y)) for y in (least, most))
    # what is not there goes to a page that no sequence holds
    spare = torch.ones(s["bounds"].shape[0], dtype=torch.int64, device=lens.device)
    spare = spare.index_fill_(0, s["table"].clamp(min=0).long().reshape(-1), 0).argmax()
    at = torch.where(here, ids, spare)
    s["bounds"][at] = torch.stack(_outwards(least, most, c), 3)


def _power(e):
    """2^e of whole numbers in [-126, 127], exactly."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_columns(s, q):
    c = s["case"]
    P, lens, k = c["page"], s["lens"].long(), c["pages"]
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    ids = s["table"].clamp(min=0).long()
    least, most = (s["bounds"][ids][:, :, :, i].float().permute(0, 2, 3, 1) for i in range(2))  # [B, H, D, N]
    e = (torch.frexp(q.abs().amax(-1, keepdim=True))[1] - 1).clamp(-100, 100)
    whole = (q * _power(6 - e)).round().clamp(-127.0, 127.0)
    x = (whole.clamp(min=0) @ most + whole.clamp(max=0) @ least) * _power(e - 6)
    G = c["q_heads"] // c["kv_heads"]
    live = (torch.arange(s["max_q"], device=lens.device)[None, :] < n[:, None])[:, None, :].expand(-1, G, -1)
    x = torch.where(live.reshape(live.shape[0], 1, -1, 1), x, torch.full_like(x, -math.inf)).amax(2)
    x = x * s["k_scales"][ids].permute(0, 2, 1)
    pages = (lens + P - 1) // P
    pages = torch.where(n > 0, pages, torch.zeros_like(pages))[:, None, None]
    j = torch.arange(ids.shape[1], device=lens.device)[None, None, :]
    own_first = torch.minimum((lens - n).clamp(min=0)[:, None, None] // P, pages - 1)
    x = torch.where((j == 0) | (j >= own_first), torch.full_like(x, math.inf), x)
    x = torch.where(j >= pages, torch.full_like(x, -math.inf), x)
    order = torch.sort(x, dim=2, descending=True, stable=True)[1][:, :, :k]
    order = torch.nn.functional.pad(order, (0, k - order.shape[2]), value=0)
    slot = torch.arange(k, device=lens.device)[None, None, :]
    far = torch.full_like(order, 1 << 30)
    order = torch.sort(torch.where(slot < pages, order, far), dim=2)[0]
    return torch.where(order == 1 << 30, torch.full_like(order, -1), order).to(torch.int32)


def _plain_select(s):
    c = s["case"]
    P, lens = c["page"], s["lens"].long()
    _plain_bounds(s, c)
    q, place = _rows_apart(s, c)
    columns = _plain_columns(s, q)
    B, H, k = columns.shape
    col = columns.long().clamp(min=0)
    ids = torch.gather(s["table"].long()[:, None, :].expand(B, H, -1), 2, col).clamp(min=0)
    heads = torch.arange(H, device=lens.device)[None, :, None].expand_as(ids)

    def values(name):
        x = _as_float(s[name + "_codes"].view(torch.uint8)[ids, heads], c) * s[name + "_scales"][ids, heads][..., None, None]
        return x.reshape(B, H, k * P, c["head_dim"])

    t = (col[..., None] * P + torch.arange(P, device=lens.device)).reshape(B, H, k * P)
    there = (columns >= 0)[..., None].expand(B, H, k, P).reshape(B, H, k * P) & (t < lens[:, None, None])
    out, lse = _attend(q, values("k"), values("v"), place, torch.where(there, t, torch.full_like(t, -1)), s, c)
    return {"bounds": s["bounds"], "columns": columns, "out": out, "lse": lse}


_RUN_PLAIN = {"rotate": _plain_rotate, "share": _plain_share, "select": _plain_select}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "share": _exact_share, "select": _exact_select}[case["op"]](s, dict(case))


def _held(s, name, ids, c, heads):
    """Values of whole pages in 64 bits, page after page: [heads, tokens, D]."""
    raw = s[name + "_codes"].view(torch.uint8)[ids][:, heads].contiguous().view(TORCH_CODE[c["code"]])
    x = raw.float().double() * s[name + "_scales"][ids][:, heads].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, c["head_dim"])


def _e4m3(y):
    """The nearest number with a sign, 3 bits behind the point and exponents from -6 up; ties to even."""
    exponent = torch.frexp(y)[1].clamp(min=-5) - 4
    unit = torch.ldexp(torch.ones_like(y), exponent)
    return torch.round(y / unit) * unit


# Codes and rotated keys are defined in steps of 32 bits, so that equal inputs give equal codes:
# each step is taken in 64 bits here and rounded where the definition says.

def _r32(x):
    return x.float().double()


def _exact_scale(largest, c):
    unit = float(torch.tensor(1.0 / QMAX[c["code"]], dtype=torch.float32))
    return torch.where(largest > 0, _r32(largest * unit).clamp(SMALLEST, LARGEST), torch.zeros_like(largest))


def _exact_codes(x, c):
    top = QMAX[c["code"]]
    y = _r32(x).clamp(-top, top)
    return y.round() if c["code"] == "int8" else _e4m3(y)


def _over(a, b):
    """a / b rounded to 32 bits, 0 where b is 0."""
    return torch.where(b > 0, _r32(a / torch.where(b > 0, b, torch.ones_like(b))), torch.zeros_like(b))


def _exact_page(x, c, before, old):
    """One page's values [tokens, D]: `old` codes held at the scale `before`, then the values x."""
    before = torch.tensor(before, dtype=torch.float64, device=x.device)
    scale = torch.maximum(before, _exact_scale(x.abs().amax(), c)) if x.numel() else before
    new = _exact_codes(x * _over(torch.ones_like(scale), scale), c) * scale
    if scale > before:
        old = _exact_codes(old * _over(before, scale), c)
    return torch.cat([old * scale, new])


def _exact_pages(x, c):
    """Rows [tokens, H, D] quantised into pages that start empty."""
    P, (m, H, D) = c["page"], x.shape
    y = torch.zeros((_pages(m, P) * P, H, D), dtype=torch.float64, device=x.device)
    y[:m] = x
    y = y.reshape(-1, P, H, D)
    scale = _exact_scale(y.abs().amax((1, 3), keepdim=True), c)
    return (_exact_codes(y * _over(torch.ones_like(scale), scale), c) * scale).reshape(-1, H, D)[:m]


def _exact_turned(x, s, c, b, first):
    """Rows [n, heads, D] of sequence b, the first of them at token `first`, pair by pair."""
    n, dim = x.shape[0], c["dim"]
    begin = int(s["cu"][b])
    y = x.double()
    for i in range(dim // 2):
        if s["positions"] is None:
            p = torch.arange(first, first + n, device=x.device)
        else:
            p = s["positions"][begin:begin + n, s["axis"][i]].long()
        cos, sin = s["turns"].double()[p, i].unbind(1)
        at = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + dim // 2)
        u, v = x[:, :, at[0]].double(), x[:, :, at[1]].double()
        y[:, :, at[0]] = _r32(_r32(u * cos[:, None]) - _r32(v * sin[:, None]))
        y[:, :, at[1]] = _r32(_r32(v * cos[:, None]) + _r32(u * sin[:, None]))
    return y


def _exact_rotate(s, c):
    lens, counts, P = _lengths(c), _counts(c), c["page"]
    H, cu, got = c["kv_heads"], s["cu"].tolist(), {}
    for n in ("k", "v"):
        value = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
        for b, (t, m) in enumerate(zip(lens, counts)):
            rows, off = s[n][cu[b]:cu[b + 1]].double(), t % P
            if n == "k":
                rows = _exact_turned(s[n][cu[b]:cu[b + 1]], s, c, b, t)
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
    q = torch.cat([_exact_turned(s["q"][cu[b]:cu[b + 1]], s, c, b, lens[b]) for b in range(c["batch"])])
    return {"k": got["k"], "v": got["v"], "q": q, "lens": None}


def _exact_rows(q, k, v, t, place, scale):
    """Attention of rows [m, D] at the positions `place` over tokens numbered t, in 64 bits."""
    x = (q.double() @ k.T) * scale
    x.masked_fill_(t[None, :] > place[:, None], -math.inf)
    z = torch.logsumexp(x, 1)
    p = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
    return p @ v, z


def _exact_results(s):
    return (torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"),
            torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda"))


def _exact_share(s, c):
    lens, counts, P = _lengths(c), _counts(c), c["page"]
    G, first = c["q_heads"] // c["kv_heads"], 0
    out, lse = _exact_results(s)
    for b, (length, m) in enumerate(zip(lens, counts)):
        t = torch.arange(length, device="cuda")
        place = torch.arange(length - m, length, device="cuda")
        ids = s["table"][b, :_pages(length, P)].long()
        for h in range(c["kv_heads"] if length else 0):
            k, v = (_held(s, n, ids, c, slice(h, h + 1))[0, :length] for n in ("k", "v"))
            for a in range(h * G, h * G + G):
                out[first:first + m, a], lse[first:first + m, a] = _exact_rows(
                    s["q"][first:first + m, a], k, v, t, place, 1.0 / math.sqrt(c["head_dim"]))
        first += m
    return {"out": out, "lse": lse}


def _exact_score(q, codes, scale, c):
    """The score of pages for rows [m, D]: codes a list of the pages' tokens [tokens, D] in 64 bits."""
    least = torch.stack([x.amin(0) for x in codes])
    most = torch.stack([x.amax(0) for x in codes])
    if c["code"] == "e4m3":
        unit = torch.full_like(least, 448)
        least, most = torch.floor(least * 127 / unit), torch.ceil(most * 127 / unit)
    best = torch.full((len(codes),), -math.inf, dtype=torch.float64, device=q.device)
    for row in q.double():
        e = min(max(math.frexp(float(row.abs().max()))[1] - 1, -100), 100)
        n = torch.round(row * 2.0 ** (6 - e)).clamp(-127, 127)
        best = torch.maximum(best, torch.maximum(n * least, n * most).sum(1) * 2.0 ** (e - 6))
    return best.float() * scale  # a product of 32-bit numbers: rounded once


def _exact_select(s, c):
    lens, counts, P = _lengths(c), _counts(c), c["page"]
    H, G, first = c["kv_heads"], c["q_heads"] // c["kv_heads"], 0
    out, lse = _exact_results(s)
    for b, (length, m) in enumerate(zip(lens, counts)):
        pages = _pages(length, P)
        ids = s["table"][b, :pages].long()
        for h in range(H if pages else 0):
            raw = s["k_codes"].view(torch.uint8)[ids, h].contiguous().view(TORCH_CODE[c["code"]]).float().double()
            codes = list(raw)
            codes[-1] = codes[-1][:length - (pages - 1) * P]
            rows = s["q"][first:first + m, h * G:h * G + G]
            if pages > c["pages"]:
                score = _exact_score(rows.reshape(-1, c["head_dim"]), codes, s["k_scales"][ids, h], c)
                kept = sorted({0} | set(range(max(length - m, 0) // P, pages)))
                others = sorted(set(range(pages)) - set(kept))
                score = score[torch.tensor(others, device="cuda")]
                best = torch.argsort(-score, stable=True)[:c["pages"] - len(kept)].tolist()
                kept = sorted(kept + [others[i] for i in best])
            else:
                kept = list(range(pages))
            at = torch.tensor(kept, device="cuda")
            t = (at[:, None] * P + torch.arange(P, device="cuda")[None, :]).reshape(-1)
            there = t < length
            k, v = (_held(s, n, ids[at], c, slice(h, h + 1))[0, there] for n in ("k", "v"))
            place = torch.arange(length - m, length, device="cuda")
            for a in range(G):
                out[first:first + m, h * G + a], lse[first:first + m, h * G + a] = _exact_rows(
                    rows[:, a], k, v, t[there], place, 1.0 / math.sqrt(c["head_dim"]))
        first += m
    return {"bounds": None, "columns": None, "out": out, "lse": lse}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(k)) for k in range(6)]:
        print(case, work(case))
