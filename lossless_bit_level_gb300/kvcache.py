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

The pages of all sequences come from one pool; the host knows every length, and what it
sends goes through pinned memory, so no call waits for the GPU (``check`` does). The host's
part of a call is Python that a graph cannot capture; the package's own calls can be. All
arithmetic is in the library's kernels (``ibp_kv_append``,
``ibp_kv_read``, ``ibp_kv_attention``, ``ibp_kv_evict``); this module only hands out pages
and buffers and orders launches on the current stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import KVCache, kv_append, kv_attention, kv_attention_scratch_bytes, kv_evict, \
    kv_evict_scratch_bytes, kv_read

_CODES = {"int8": torch.int8}
if hasattr(torch, "float8_e4m3fn"):
    _CODES["e4m3"] = torch.float8_e4m3fn


class DecodeCache:
    """Cache of one attention layer for ``batch`` sequences.

    n_pages pages of page_tokens tokens are shared by the sequences, each of which holds at
    most max_tokens. ``track_weights`` keeps the probabilities that ``attend`` gave each
    token, summed over steps with the factor ``decay``, for ``evict`` to go by."""

    def __init__(self, n_pages: int, batch: int, n_heads: int, head_dim: int, max_tokens: int,
                 page_tokens: int = 64, code: str = "int8", track_weights: bool = True,
                 decay: float = 1.0, device: torch.device | str = "cuda"):
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

    def append(self, k: torch.Tensor, v: torch.Tensor, counts=None) -> None:
        """Rows [n, heads, head_dim] behind what the sequences hold: counts[b] of them to
        sequence b, one sequence after another (None: the same number each)."""
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
            kv_append(now, k, v, cu=None if each is None else self._offsets(counts),
                      new_lens=later.lens, status=self.status)
            now.lens.copy_(later.lens)
        self.lengths, self._pages = after, pages

    def load(self, k_store, v_store, counts=None) -> None:
        """Append the rows of two compressed tensors (``offload.CompressedTensor``, a row a
        token of n_heads * head_dim 16- or 32-bit floats): decoded on the GPU, then
        quantised into the pages."""
        from . import BF16, FP16, FP32
        kinds = {BF16: torch.bfloat16, FP16: torch.float16, FP32: torch.float32}
        rows = []
        for store in (k_store, v_store):
            out = store.empty_like(self.device)
            store.decompress_into(out)
            rows.append(out.view(kinds[store.dtype]).view(store.n_rows, self.cache.n_heads,
                                                          self.cache.head_dim))
        self.append(rows[0], rows[1], counts)

    def attend(self, q: torch.Tensor, scale: float, counts=None,
               lse: torch.Tensor | None = None) -> torch.Tensor:
        """softmax(scale * q k) v of query rows [n, q_heads, head_dim], counts[b] of them the
        last tokens of sequence b. Adds their probabilities to the tokens' weights."""
        each, counts = counts, self._counts(counts, q.shape[0])
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        most, track = max(counts, default=0), self.weights is not None
        scratch = self._workspace(kv_attention_scratch_bytes(
            self.cache, q.shape[0], most, q.shape[1], track))
        kv_attention(self.cache, q, out, scale, scratch,
                     cu_q=None if each is None else self._offsets(counts), max_q=most, lse=lse,
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
        for p in self._pages:
            self._free.extend(p)
        if into is not None:
            self.weights, self._weights_after = into, self.weights
        self._handles, self._pages, self.lengths = [later, now], pages, kept

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
