"""An 8-bit paged key/value cache that a decoding loop keeps on the GPU, next to the
losslessly compressed K/V rows that stay in host memory.

"Reducing the GPU Memory Bottleneck with Lossless Compression for ML -- Extended",
technical summary, "System integration": offloaded inference keeps the KV cache as rows of
tokens in host memory and brings them over compressed. What attention reads every step has
to be on the GPU; this class holds it there in 8 bits an element (one scale for each page
and head), attends over it, and keeps it within a budget of tokens by dropping those that
were attended least:

    host rows (IBP slots) --load--> pages <--append-- new tokens
                                      |  attend (adds up each token's probabilities)
                                      +--evict--> fewer pages --read--> rows again

Rows may be rotated by their positions on the way in (``append`` and ``load`` with a
``KVRotation``, their queries with them). Sequences that begin alike hold the pages of their
beginning once (``share``) and ``attend`` goes over it once for all of them. With
``track_bounds`` a step may attend over a few pages only, those that a cheap score finds for
each sequence and head (``attend`` with ``pages``).

The pages of all sequences come from one pool; the host knows every length, and what it
sends goes through pinned memory, so no call waits for the GPU (``check`` does). The host's
part of a call is Python that a graph cannot capture; the package's own calls can be. All
arithmetic is in the library's kernels (``ibp_kv_append`` and ``ibp_kv_append_rotated``,
``ibp_kv_read``, ``ibp_kv_attention``, ``.._shared`` and ``.._selected``, ``ibp_kv_bounds``,
``ibp_kv_select``, ``ibp_kv_evict``); this module only hands out pages
and buffers and orders launches on the current stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import KVCache, KVRotation, kv_append, kv_append_rotated, kv_attention, \
    kv_attention_scratch_bytes, kv_attention_selected, kv_attention_selected_scratch_bytes, \
    kv_attention_shared, kv_attention_shared_scratch_bytes, kv_bounds, kv_evict, \
    kv_evict_scratch_bytes, kv_read, kv_select, kv_select_scratch_bytes

_CODES = {"int8": torch.int8}
if hasattr(torch, "float8_e4m3fn"):
    _CODES["e4m3"] = torch.float8_e4m3fn


class DecodeCache:
    """Cache of one attention layer for ``batch`` sequences.

    n_pages pages of page_tokens tokens are shared by the sequences, each of which holds at
    most max_tokens. ``track_weights`` keeps the probabilities that ``attend`` gave each
    token, summed over steps with the factor ``decay``, for ``evict`` to go by.
    ``track_bounds`` keeps the pages' bounds that ``attend`` selects pages by."""

    def __init__(self, n_pages: int, batch: int, n_heads: int, head_dim: int, max_tokens: int,
                 page_tokens: int = 64, code: str = "int8", track_weights: bool = True,
                 decay: float = 1.0, device: torch.device | str = "cuda",
                 track_bounds: bool = False):
        if code not in _CODES:
            raise ValueError(f"code must be one of {sorted(_CODES)}")
        shape = (n_pages, n_heads, page_tokens, head_dim)
        self.page_tokens, self.decay, self.device = page_tokens, decay, torch.device(device)
        cols = -(-max_tokens // page_tokens)
        zeros = lambda *s, dtype: torch.zeros(s, dtype=dtype, device=self.device)  # noqa: E731
        self._pools = tuple(zeros(*shape, dtype=torch.uint8).view(_CODES[code]) for _ in range(2)) + \
            tuple(zeros(n_pages, n_heads, dtype=torch.float32) for _ in range(2))
        self.max_tokens = cols * page_tokens
        self.lengths = [0] * batch             # as the host knows them
        self._seen = [0] * batch               # tokens so far, those that were evicted among them
        self._pages: list[list[int]] = [[] for _ in range(batch)]
        self._free = list(range(n_pages - 1, -1, -1))
        # two tables and lengths: a call reads one and writes the other
        self._handles = [KVCache(*self._pools, torch.full((batch, cols), -1, dtype=torch.int32,
                                                          device=self.device),
                                 zeros(batch, dtype=torch.int32)) for _ in range(2)]
        self.weights = None
        if track_weights:
            self.weights = zeros(batch, n_heads, self.max_tokens, dtype=torch.float32)
            self._weights_after = torch.zeros_like(self.weights)
        self.bounds = zeros(*self._handles[0].bounds_shape, dtype=torch.int8) if track_bounds else None
        self._groups: list[tuple[int, int, int]] = []  # sequences [first, past) and their shared tokens
        self._group_tensors = None
        self.status = zeros(1, dtype=torch.int32)

    @property
    def cache(self) -> KVCache:
        """Handle of the cache as it is now (for the calls of the package)."""
        return self._handles[0]

    @property
    def pages_free(self) -> int:
        return len(self._free)

    def _workspace(self, n: int) -> torch.Tensor:
        """Scratch of one call: PyTorch's allocator takes it back when the call is in the stream,
        so that the layers of a model share what the largest of their calls needs."""
        return torch.empty(max(n, 16), dtype=torch.uint8, device=self.device)

    def _counts(self, counts, n: int) -> list[int]:
        batch = len(self.lengths)
        if counts is None:
            if n % batch:
                raise ValueError(f"{n} rows do not divide among {batch} sequences: pass counts")
            return [n // batch] * batch
        counts = [int(c) for c in counts]
        if len(counts) != batch or min(counts, default=0) < 0 or sum(counts) != n:
            raise ValueError(f"counts must be {batch} numbers that add up to {n}")
        return counts

    def _pinned(self, numbers) -> torch.Tensor:
        # a copy from pageable memory waits for the stream once it is larger than 64 KB
        return torch.tensor(numbers, dtype=torch.int32, pin_memory=self.device.type == "cuda")

    def _offsets(self, counts: list[int]) -> torch.Tensor:
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        return self._pinned(cu).to(self.device, non_blocking=True)

    def _take(self, need: list[int]) -> list[list[int]]:
        if sum(need) > len(self._free):
            raise RuntimeError(f"{sum(need)} pages are needed and {len(self._free)} are free")
        return [[self._free.pop() for _ in range(n)] for n in need]

    @contextlib.contextmanager
    def _pages_for(self, need: list[int]):
        """Pages of the pool, need[b] for each sequence, which go back to it if what is done
        with them raises (a call that refuses its arguments, no memory)."""
        taken = self._take([max(n, 0) for n in need])
        try:
            yield taken
        except BaseException:
            self._free.extend(reversed([p for pages in taken for p in pages]))
            raise

    def _write_table(self, handle: KVCache, rows: list[list[int]]) -> None:
        # the columns in use; what a table holds past a sequence's pages is never read
        cols = max((len(r) for r in rows), default=0)
        if cols:
            host = self._pinned([r + [-1] * (cols - len(r)) for r in rows])
            handle.table[:, :cols].copy_(host, non_blocking=True)

    def _numbers(self, counts: list[int], axes: int) -> torch.Tensor | None:
        """Positions [n, axes] of new rows: each its token's number among all that its sequence
        was given. None while a token's place in the cache says that; where tokens were evicted
        their places are taken by later ones, and what is kept stays rotated by its own number."""
        if self._seen == self.lengths:
            return None
        host = torch.empty((sum(counts), axes), dtype=torch.int32, pin_memory=self.device.type == "cuda")
        at = 0
        for seen, n in zip(self._seen, counts):
            host[at:at + n] = torch.arange(seen, seen + n, dtype=torch.int32)[:, None]
            at += n
        return host.to(self.device, non_blocking=True)

    def append(self, k: torch.Tensor, v: torch.Tensor, counts=None,
               rotation: KVRotation | None = None, positions: torch.Tensor | None = None,
               q: torch.Tensor | None = None) -> torch.Tensor | None:
        """Rows [n, heads, head_dim] behind what the sequences hold: counts[b] of them to
        sequence b, one sequence after another (None: the same number each). With ``rotation``
        keys are rotated on the way, by ``positions`` (int32 [n, axes]; None: the tokens'
        numbers among all that their sequences were given, evicted ones counted), and so are the
        query rows ``q`` of the same tokens, which are returned."""
        if rotation is None and (q is not None or positions is not None):
            raise ValueError("positions and q go with a rotation")
        each, counts = counts, self._counts(counts, k.shape[0])
        after = [n + c for n, c in zip(self.lengths, counts)]
        if max(after, default=0) > self.max_tokens:
            raise ValueError(f"a sequence would hold {max(after)} of {self.max_tokens} tokens")
        need = [-(-n // self.page_tokens) - len(p) for n, p in zip(after, self._pages)]
        now, later = self._handles
        with self._pages_for(need) as new:
            pages = [p + q for p, q in zip(self._pages, new)]
            if any(need):
                self._write_table(now, pages)
            cu = None if each is None else self._offsets(counts)
            turned = None
            if rotation is None:
                kv_append(now, k, v, cu=cu, new_lens=later.lens, status=self.status)
            else:
                if positions is None:
                    positions = self._numbers(counts, rotation.axes)
                if q is not None:
                    turned = torch.empty_like(q, memory_format=torch.contiguous_format)
                kv_append_rotated(now, k, v, rotation, positions=positions, q=q, q_out=turned, cu=cu,
                                  new_lens=later.lens, status=self.status)
            before = now.lens.clone() if self.bounds is not None else None
            now.lens.copy_(later.lens)
        self._seen = [n + c for n, c in zip(self._seen, counts)]
        self.lengths, self._pages = after, pages
        if before is not None:
            kv_bounds(now, self.bounds, begin=before, status=self.status)
        return turned

    def share(self, src: int, sequences) -> int:
        """Let ``sequences``, which are empty and follow src one after another, begin with the
        whole pages that sequence src holds; returns how many tokens that is (what src holds
        behind them they do not get). ``attend`` goes over these pages once for all of them where
        the cache tracks no weights (``track_weights=False``); with weights, which are each
        sequence's own and begin at 0, every sequence is gone over by itself."""
        wanted = list(sequences)
        if wanted != list(range(src + 1, src + 1 + len(wanted))) or not wanted or \
                not 0 <= src < len(self.lengths) or wanted[-1] >= len(self.lengths):
            raise ValueError("sequences that share follow the first of them one after another")
        if any(self.lengths[b] for b in wanted):
            raise ValueError("a sequence that takes shared pages is empty")
        if any(first < wanted[-1] + 1 and src < past for first, past, _ in self._groups):
            raise ValueError("a sequence shares one beginning")
        tokens = self.lengths[src] // self.page_tokens * self.page_tokens
        begin = self._pages[src][:tokens // self.page_tokens]
        if not begin:
            return 0
        pages = list(self._pages)
        for b in wanted:
            pages[b] = list(begin)
        now = self.cache
        self._write_table(now, pages)
        now.lens[wanted[0]:wanted[-1] + 1] = tokens  # (a fill: nothing is sent)
        for b in wanted:
            self.lengths[b] = tokens
            # the least number past all of the shared tokens: places keep the tokens' order in
            # every head, and src holds so many behind them
            self._seen[b] = self._seen[src] - (self.lengths[src] - tokens)
        self._pages = pages
        self._groups = sorted(self._groups + [(src, wanted[-1] + 1, tokens)])
        self._group_tensors = None
        return tokens

    def _shared(self):
        """Offsets of the groups and their shared tokens, on the device; sequences between groups
        are groups that share nothing."""
        if self._group_tensors is None:
            offsets, prefix = [0], []
            for first, past, tokens in self._groups:
                if first > offsets[-1]:
                    offsets.append(first)
                    prefix.append(0)
                offsets.append(past)
                prefix.append(tokens)
            self._group_tensors = tuple(self._pinned(x).to(self.device, non_blocking=True)
                                        for x in (offsets, prefix))
        return self._group_tensors

    def load(self, k_store, v_store, counts=None, rotation: KVRotation | None = None,
             positions: torch.Tensor | None = None) -> None:
        """Append the rows of two compressed tensors (``offload.CompressedTensor``, a row a
        token of n_heads * head_dim 16- or 32-bit floats): decoded on the GPU, then
        quantised into the pages, with ``rotation`` rotated before that."""
        from . import BF16, FP16, FP32
        kinds = {BF16: torch.bfloat16, FP16: torch.float16, FP32: torch.float32}
        rows = []
        for store in (k_store, v_store):
            out = store.empty_like(self.device)
            store.decompress_into(out)
            rows.append(out.view(kinds[store.dtype]).view(store.n_rows, self.cache.n_heads,
                                                          self.cache.head_dim))
        self.append(rows[0], rows[1], counts, rotation=rotation, positions=positions)

    def attend(self, q: torch.Tensor, scale: float, counts=None,
               lse: torch.Tensor | None = None, pages: int | None = None) -> torch.Tensor:
        """softmax(scale * q k) v of query rows [n, q_heads, head_dim], counts[b] of them the
        last tokens of sequence b. Adds their probabilities to the tokens' weights. With
        ``pages`` a sequence and head attends over so many of its pages: the first, the rows'
        own, and those of the highest scores (needs ``track_bounds``; adds no weights).
        Without weights to add to, beginnings that sequences share are gone over once."""
        each, counts = counts, self._counts(counts, q.shape[0])
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        most, track = max(counts, default=0), self.weights is not None
        cu = None if each is None else self._offsets(counts)
        if pages is not None:
            if self.bounds is None:
                raise RuntimeError("pages are selected by bounds, which this cache does not track")
            columns = torch.empty((len(self.lengths), self.cache.n_heads, pages), dtype=torch.int32,
                                  device=self.device)
            kv_select(self.cache, self.bounds, q, columns,
                      self._workspace(kv_select_scratch_bytes(self.cache)), cu_q=cu, max_q=most,
                      status=self.status)
            scratch = self._workspace(kv_attention_selected_scratch_bytes(
                self.cache, q.shape[0], most, q.shape[1], pages))
            kv_attention_selected(self.cache, columns, q, out, scale, scratch, cu_q=cu, max_q=most,
                                  lse=lse, status=self.status)
            return out
        if self._groups and not track:
            offsets, prefix = self._shared()
            rows = max(sum(counts[first:past]) for first, past, _ in self._groups)
            scratch = self._workspace(kv_attention_shared_scratch_bytes(
                self.cache, q.shape[0], most, q.shape[1], prefix.numel(), rows))
            kv_attention_shared(self.cache, q, out, scale, scratch, offsets, prefix, rows, cu_q=cu,
                                max_q=most, lse=lse, status=self.status)
            return out
        scratch = self._workspace(kv_attention_scratch_bytes(
            self.cache, q.shape[0], most, q.shape[1], track))
        kv_attention(self.cache, q, out, scale, scratch,
                     cu_q=cu, max_q=most, lse=lse,
                     weights=self.weights, weights_in=self.weights, decay=self.decay,
                     status=self.status)
        return out

    def evict(self, budget: int, recent: int) -> None:
        """Keep ``budget`` tokens of every longer sequence and head: the last ``recent`` and
        those that were attended most. Needs free pages for what is kept; the old ones are
        free afterwards (calls on the same stream come after this one)."""
        if self.weights is None:
            raise RuntimeError("evict goes by the weights, which this cache does not track")
        now, later = self._handles
        kept = [min(n, budget) for n in self.lengths]
        with self._pages_for([-(-n // self.page_tokens) for n in kept]) as pages:
            self._write_table(later, pages)
            scratch = self._workspace(kv_evict_scratch_bytes(now, budget))
            into = self._weights_after if budget <= self.max_tokens else None
            kv_evict(now, self.weights, budget, recent, later, scratch, new_weights=into,
                     status=self.status)
        self._free.extend(dict.fromkeys(p for of_one in self._pages for p in of_one))  # shared ones once
        self._groups, self._group_tensors = [], None  # every sequence has its own now
        if into is not None:
            self.weights, self._weights_after = into, self.weights
        self._handles, self._pages, self.lengths = [later, now], pages, kept
        if self.bounds is not None:
            kv_bounds(later, self.bounds, status=self.status)

    def read(self, dtype: torch.dtype = torch.bfloat16) -> tuple[torch.Tensor, torch.Tensor]:
        """Every sequence's tokens as rows [batch, longest, heads, head_dim] (zeros past the
        length): rows that the codec's calls take."""
        shape = (len(self.lengths), max(max(self.lengths, default=0), 1), self.cache.n_heads,
                 self.cache.head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=self.device) for _ in range(2))
        kv_read(self.cache, k, v, status=self.status)
        return k, v

    def check(self) -> None:
        """Wait for the GPU and raise if a kernel recorded an error."""
        code = int(self.status.item())
        if code:
            from . import IBPError
            raise IBPError(code, "key/value cache")
