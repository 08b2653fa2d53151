/*
 * ibp.h -- C ABI of the GB300 (sm_103a) Invariant Bit Packing codec.
 *
 * Method: "Reducing the GPU Memory Bottleneck with Lossless Compression for ML --
 * Extended" (Kamath, Krishnamurthy, Canini, Peter), technical summary:
 *   - "Core algorithm", preprocessing: find the bit positions of the element word
 *     that hold one value in at least a fraction T of a sample, keep them as a
 *     fixed-size mask + bitval in GPU memory, reuse them for the whole dataset;
 *   - "Core algorithm", compression: per fixed-size block, test the invariant
 *     positions against bitval; on a match strip them and close the gaps; mark
 *     each block with a participation bit; run on the GPU over zero-copy memory;
 *   - "Core algorithm", decompression: a warp stages a contiguous compressed
 *     segment in shared memory, prefix-scans block sizes with warp primitives to
 *     find each block's bit offset, and reinserts the invariant bits;
 *   - "System integration", PCIe transfer compression: one fixed-size buffer per
 *     tensor of which only the compressed part is read, plus a GPU-resident
 *     bitmask of which tensors are compressed.
 *
 * Conventions shared by every call
 *   - A "row" is the unit stored in one slot (a feature vector, an embedding
 *     row, a weight row, a token's K or V). Rows are row_elems little-endian
 *     element words of w bits: w = 32 (IBP_FP32), 16 (IBP_FP16, IBP_BF16) or 8
 *     (IBP_W8).
 *     Only bit patterns are handled: +-0, denormals, Inf and NaN payloads are
 *     ordinary words and always round-trip exactly.
 *   - block_elems B must be 32 or 64; 1 <= row_elems <= 2^20. A row is cut into
 *     nb = ceil(row_elems / B) blocks; when B does not divide row_elems the last
 *     block holds the remaining elements (its own participation bit, sized
 *     1 + len*m or 1 + len*w bits), and the row must then be a multiple of 16
 *     bytes long (row_elems * w / 8 % 16 == 0).
 *   - Slot r of a store starts at slots + r*slot_bytes; slot_bytes is at least
 *     ibp_slot_bytes() (the raw row rounded up to 16 bytes) and a multiple of 16.
 *   - Stream format of a compressed row (bit i = bit i%32 of little-endian 32-bit
 *     word i/32): nb participation bits, then each block in order, either one
 *     field of m = w - popcount(mask) bits per element (the element's
 *     non-invariant bits, ascending) or the raw words. A row is stored compressed
 *     iff 4*ceil(bits/32) < raw bytes, where bits = sum_b (1 + len_b*m) or
 *     (1 + len_b*w), len_b = B except for a shorter last block.
 *   - Bitmask: bit r of a store is bit r%32 of 32-bit word r/32.
 *   - Ownership: the caller owns and allocates every buffer; the library
 *     allocates nothing, keeps no per-call state and never synchronises a stream
 *     except where stated. Pointers named d_* must be device memory. rows and
 *     slots may be device memory or page-locked host memory registered with CUDA
 *     (read and written zero-copy by the kernels); pageable host memory is
 *     rejected. rows, slots and out must be 16-byte aligned.
 *   - Every compute call is asynchronous on stream s (0 = legacy default stream)
 *     and may be captured in a CUDA graph once the argument checks pass.
 *
 * Return codes: IBP_OK (0) or a negative code found before anything is launched.
 * Errors a kernel detects are written to *d_status (when it is non-null) with an
 * atomic compare-and-swap from 0, so the first error wins; the caller zeroes
 * *d_status before the call. No kernel traps, asserts or waits without bound.
 */
#ifndef IBP_H
#define IBP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *ibp_stream_t; /* same object as cudaStream_t */

/* Element word widths: 32 bits (FP32), 16 bits (FP16, BF16), 8 bits (IBP_W8: FP8
 * E4M3/E5M2, int8, uint8 -- only the width matters, bit patterns are opaque). */
typedef enum { IBP_FP32 = 0, IBP_FP16 = 1, IBP_BF16 = 2, IBP_W8 = 3 } ibp_dtype;

enum {
  IBP_OK = 0,
  IBP_ERR_ARG = -1,         /* null/misaligned/pageable pointer, bad size, T outside [0,1] */
  IBP_ERR_DTYPE = -2,       /* dtype not one of ibp_dtype */
  IBP_ERR_UNSUPPORTED = -3, /* block size or row length the kernels do not handle */
  IBP_ERR_CUDA = -4,        /* a CUDA call or launch failed */
  IBP_ERR_INDEX = -5,       /* (device) gather index outside [0, n_rows) */
  IBP_ERR_CORRUPT = -6,     /* (device) participation bits describe an impossible stream */
  IBP_ERR_META = -7,        /* (device) *d_meta disagrees with the dtype/block_elems passed */
  IBP_ERR_TIMEOUT = -8      /* (device) a bounded wait inside a kernel ran out; output incomplete */
};

/* Metadata: the fixed-size mask/bitval pair of the preprocessing stage.
 * Plain data (16 bytes); the caller may copy or serialise it. mask has a 1 at
 * every invariant bit position; bitval holds their values and is 0 elsewhere.
 * dtype == IBP_META_INVALID marks metadata that ibp_meta_finalize refused to build
 * (every call given it reports IBP_ERR_META). */
#define IBP_META_INVALID 0xFFFFFFFFu

typedef struct {
  uint32_t mask;
  uint32_t bitval;
  uint32_t dtype;       /* ibp_dtype */
  uint32_t block_elems; /* B */
} ibp_meta;

/* Store statistics written by ibp_query / ibp_query_async. */
typedef struct {
  int64_t n_rows;
  int64_t n_compressed; /* rows whose bitmask bit is 1 */
  int64_t raw_bytes;    /* n_rows * row_elems * w/8 */
  int64_t stored_bytes; /* sum over rows: 4*ceil(bits/32) if compressed, else raw row bytes */
  int64_t total_bits;   /* sum over rows of the size formula, compressed or not */
} ibp_stats;

/* Human-readable name of a return/status code (static string). */
const char *ibp_status_string(int code);

/* Bytes of one slot ("System integration": every tensor gets one fixed-size buffer
 * whose leading, compressed part is all that is read; the buffer must hold the row
 * raw, since a row that does not shrink is stored as it is): row_elems * w/8
 * rounded up to 16 (the kernels move 16-byte vectors). row_elems <= 0: IBP_ERR_ARG;
 * unknown dtype: IBP_ERR_DTYPE. Pure host arithmetic, no CUDA call. */
int ibp_slot_bytes(int64_t row_elems, int dtype, int64_t *slot_bytes);

/* Bytes of device scratch ibp_build_meta needs ("Core algorithm", preprocessing:
 * the metadata follows from how often each bit position of the element word holds
 * a 1 in the sample, so the scratch holds one 64-bit count per bit position of a
 * 32-bit word: 256 bytes, whatever the input size). Host arithmetic only. */
int ibp_meta_scratch_bytes(size_t *bytes);

/* Preprocessing ("Core algorithm", preprocessing).
 * rows: n_rows x row_elems element words (device or registered host memory).
 * For every bit position j < w, counts the sampled elements whose bit j is 1; j is
 * invariant iff the majority value's count c satisfies (double)c >= T*(double)N in
 * IEEE double (N = n_rows*row_elems; a tie counts as majority value 0).
 * Writes *d_meta = {mask, bitval, dtype, block_elems}. d_scratch: device memory of
 * ibp_meta_scratch_bytes(), overwritten (no initial contents needed). */
int ibp_build_meta(const void *rows, int64_t n_rows, int64_t row_elems, int dtype, double T,
                   uint32_t block_elems, ibp_meta *d_meta, void *d_scratch, ibp_stream_t s);

/* Preprocessing ("Core algorithm", preprocessing) in two steps, for rows held in
 * several places (shards of a table on several GPUs, or batches streamed one after
 * another): the per-position counts of disjoint row sets add up.
 * ibp_meta_count: rows as for ibp_build_meta (device or registered host memory, a
 * whole number of 32-bit words, 16-byte aligned; n_rows may be 0). Overwrites
 * d_counters (32 uint64 words = 256 bytes of device memory, 8-byte aligned) with the
 * number of 1s at each bit position of the rows' 32-bit words (8- and 16-bit elements
 * are folded into their element positions by the finalize step).
 * The holders' counters are then summed by the caller (an all-reduce of the 32 words
 * across GPUs, or an elementwise add on one GPU).
 * ibp_meta_finalize: applies the threshold rule of ibp_build_meta to the summed
 * counters, n_elems (> 0) being the total number of elements counted, and writes
 * *d_meta. T outside [0, 1] or n_elems <= 0: IBP_ERR_ARG; block_elems not 32 or 64:
 * IBP_ERR_UNSUPPORTED. A counter larger than n_elems (the counters and the element
 * count do not describe the same rows, e.g. one holder's count passed with summed
 * counters) is detected on the device: *d_meta is then written with mask = bitval =
 * 0 and dtype = IBP_META_INVALID, so that every later call given it reports
 * IBP_ERR_META, and IBP_ERR_META is recorded in *d_status (nullable, device memory,
 * compare-and-swap from 0). With one holder the pair equals ibp_build_meta. Both
 * calls are asynchronous on s and allocate nothing. */
int ibp_meta_count(const void *rows, int64_t n_rows, int64_t row_elems, int dtype,
                   uint64_t *d_counters, ibp_stream_t s);
int ibp_meta_finalize(const uint64_t *d_counters, int64_t n_elems, int dtype, double T,
                      uint32_t block_elems, ibp_meta *d_meta, int32_t *d_status,
                      ibp_stream_t s);

/* ibp_build_meta for callers that cannot allocate device memory (the paper has no
 * counterpart; this is a library convenience). Same arguments, checks and result
 * as ibp_build_meta, except that the counters live in a 256-byte array built into
 * the library (kept by every GPU that loads it until the process exits) instead of
 * caller-provided scratch. Meant for code that must not call cudaMalloc when it
 * needs the metadata: a plug-in inside a framework whose allocator owns all device
 * memory, a latency-critical loop where an allocation's implicit synchronisation is
 * not allowed, a system that forbids allocation after start-up.
 * - Allocates nothing: no cudaMalloc/cudaFree and no allocating library call.
 * - The first call on a device looks up the array's device address (once per
 *   device, with that device current); make that first call before any stream
 *   capture. The address is kept together with the identity of the CUDA context it
 *   was looked up in; after a device reset (a new primary context, where the
 *   library's device code is loaded again) the next call looks it up again, so
 *   make that call, too, before any capture.
 * - The counters are cleared on stream s at the start of every call, so results
 *   never depend on an earlier call; but every call shares the one array, so calls
 *   whose kernels overlap on the GPU (e.g. on unordered streams) race and give
 *   undefined results. Order them on one stream or with events.
 * - Returns IBP_ERR_UNSUPPORTED if the counters ever needed more than the 256 bytes
 *   built in (ibp_meta_scratch_bytes() is 256 for every input size today). */
int ibp_build_meta_noalloc(const void *rows, int64_t n_rows, int64_t row_elems, int dtype,
                           double T, uint32_t block_elems, ibp_meta *d_meta, ibp_stream_t s);

/* Saving-aware metadata: a variant of preprocessing (the paper has no counterpart;
 * it follows from "Core algorithm": the threshold rule picks positions one by one,
 * but compression strips a block's invariant bits only when every one of them
 * holds in every element, so a position whose few exceptions fall in many blocks
 * can cost more than it saves).
 * Candidates: candidate 0 is the mask ibp_build_meta gives for T (M0); candidate
 * k+1 is candidate k without every position whose majority value is held by the
 * fewest elements among the positions candidate k still has (equal counts leave
 * together); the last candidate is the empty mask, so there are 1 to w+1 of them.
 * Each candidate's bitval is M0's bitval restricted to it. Each candidate is scored
 * by the bytes rows [0, n_rows) take when compressed with it: the sum over rows of
 * 4*ceil(bits/32) for a row stored compressed and the raw row bytes otherwise.
 * *d_meta receives the lowest-scoring candidate, ties going to the lower k (the
 * larger mask). With T <= 0.5 every position is in M0 and the candidates are all
 * the masks the threshold rule gives for any threshold, plus the empty mask.
 * d_candidates (nullable; device memory of IBP_MAX_MASK_CANDIDATES entries): entry
 * k receives candidate k and its score; entries past the last candidate receive
 * mask = bitval = 0 and stored_bytes = -1.
 * d_scratch: ibp_meta_select_scratch_bytes() bytes of device memory, overwritten.
 * Reads the rows twice (counting, then scoring); same argument checks and codes as
 * ibp_build_meta. */
#define IBP_MAX_MASK_CANDIDATES 33

typedef struct {
  uint32_t mask;
  uint32_t bitval;
  int64_t stored_bytes; /* score of this candidate, or -1 for an unused entry */
} ibp_mask_candidate;   /* 16 bytes */

int ibp_meta_select_scratch_bytes(size_t *bytes);

int ibp_build_meta_select(const void *rows, int64_t n_rows, int64_t row_elems, int dtype,
                          double T, uint32_t block_elems, ibp_meta *d_meta,
                          ibp_mask_candidate *d_candidates, void *d_scratch, ibp_stream_t s);

/* Compression ("Core algorithm", compression; "System integration").
 * Encodes rows [0, n_rows) into their slots with the mask/bitval in *d_meta, whose
 * dtype and block_elems must equal the ones passed. Compressed rows hold their
 * stream in the first 4*ceil(bits/32) bytes of the slot (the rest of the slot up
 * to the next 16-byte boundary is written with zeros, later bytes are untouched);
 * other rows hold their raw bytes. d_row_bitmask (ceil(n_rows/32) words) is fully
 * rewritten, bits past n_rows set to 0. d_row_bits (nullable, n_rows words)
 * receives each row's size-formula bit count. rows and slots must not overlap. */
int ibp_compress(const void *rows, int64_t n_rows, int64_t row_elems, int dtype,
                 uint32_t block_elems, const ibp_meta *d_meta, void *slots, int64_t slot_bytes,
                 uint32_t *d_row_bitmask, uint32_t *d_row_bits, int32_t *d_status,
                 ibp_stream_t s);

/* Decompress-gather ("Core algorithm", decompression; "System integration").
 * out[i] (row_elems words, device memory, rows packed back to back) receives the
 * original row d_idx[i] for i < n_idx; indices may repeat. Only the used prefix of
 * each slot is read. n_idx == 0 is a no-op. A row whose index is outside
 * [0, n_rows) or whose participation bits describe a stream that would not have
 * been stored compressed is skipped (out[i] untouched) and IBP_ERR_INDEX or
 * IBP_ERR_CORRUPT is recorded in *d_status. */
int ibp_decompress_gather(const void *slots, int64_t slot_bytes, int64_t n_rows,
                          int64_t row_elems, int dtype, uint32_t block_elems,
                          const uint32_t *d_row_bitmask, const ibp_meta *d_meta,
                          const int64_t *d_idx, int64_t n_idx, void *out, int32_t *d_status,
                          ibp_stream_t s);

/* Packed store ("System integration": compressing a GPU cache's rows raises its
 * effective capacity; the paper has no layout for it, so this one is the
 * library's). A slotted store keeps every row in a raw-size slot (a row can be
 * rewritten in place); a packed store lays rows end to end and is read only:
 *   entry i = the used prefix of slot d_sel[i] (d_sel null: row i) -- the
 *     4*ceil(bits/32) stream bytes of a compressed row, or the raw row -- rounded up
 *     to a multiple of 16 bytes, copied from the slot (stream padding included);
 *   d_offsets[i] = byte offset of entry i; d_offsets[n_sel] = total bytes
 *     (n_sel + 1 uint64 entries, device memory).
 * Entry i of the packed store is row i: its bitmask bit and bit count are the
 * source row's. Build it in three calls: ibp_pack_offsets, read d_offsets[n_sel]
 * to size the buffer, ibp_pack. */

/* Device scratch ibp_pack_offsets needs for n_sel entries (8 bytes per 4096). */
int ibp_pack_scratch_bytes(int64_t n_sel, size_t *bytes);

/* Entry offsets of a packed store of rows d_sel[0..n_sel) of a slotted store
 * described by d_row_bitmask and d_row_bits (both as written by ibp_compress;
 * row_bits is required here). A selection outside [0, n_rows) gets a 0-byte entry
 * and IBP_ERR_INDEX in *d_status. Asynchronous on s. */
int ibp_pack_offsets(const uint32_t *d_row_bitmask, const uint32_t *d_row_bits, int64_t n_rows,
                     int64_t row_elems, int dtype, const int64_t *d_sel, int64_t n_sel,
                     uint64_t *d_offsets, void *d_scratch, int32_t *d_status, ibp_stream_t s);

/* Copy the entries into packed (device or registered host memory, packed_bytes
 * long, 16-byte aligned) and write the packed store's bitmask d_pack_bitmask
 * (ceil(n_sel/32) words, fully rewritten) and, when non-null, d_pack_row_bits
 * (n_sel words). An entry whose offsets disagree with its row's size, are not
 * 16-byte aligned or leave the buffer is skipped with IBP_ERR_CORRUPT in
 * *d_status; a bad selection with IBP_ERR_INDEX. slots and packed must not
 * overlap. */
int ibp_pack(const void *slots, int64_t slot_bytes, int64_t n_rows, int64_t row_elems, int dtype,
             const uint32_t *d_row_bitmask, const uint32_t *d_row_bits, const int64_t *d_sel,
             int64_t n_sel, const uint64_t *d_offsets, void *packed, uint64_t packed_bytes,
             uint32_t *d_pack_bitmask, uint32_t *d_pack_row_bits, int32_t *d_status,
             ibp_stream_t s);

/* ibp_decompress_gather on a packed store of n_rows entries: row r is read from
 * packed + d_offsets[r], d_offsets[r+1] - d_offsets[r] bytes of it. Rows of at most
 * 32 blocks are staged whole (exactly their entry) with no header round trip. An
 * entry whose offsets are unaligned, decreasing or past packed_bytes, or too short
 * for the row its header describes, is skipped with IBP_ERR_CORRUPT. */
int ibp_decompress_gather_packed(const void *packed, uint64_t packed_bytes,
                                 const uint64_t *d_offsets, int64_t n_rows, int64_t row_elems,
                                 int dtype, uint32_t block_elems, const uint32_t *d_row_bitmask,
                                 const ibp_meta *d_meta, const int64_t *d_idx, int64_t n_idx,
                                 void *out, int32_t *d_status, ibp_stream_t s);

/* De-duplicated decompress-gather ("Core algorithm", decompression; "System
 * integration", rows in host memory moved over the host link). Same arguments and
 * result as ibp_decompress_gather: out[i] (n_idx x row_elems words, device memory)
 * is row d_idx[i]; an index outside [0, n_rows) records IBP_ERR_INDEX in *d_status
 * and leaves its output row untouched. Each distinct row of d_idx is read from its
 * slot and decoded once, straight into the output row of one position that names it
 * (the first to claim it), then copied from there to every other position that names
 * it: for skewed index lists a row crosses the host link once instead of once per
 * request. d_scratch: device memory of scratch_bytes >= the size
 * ibp_gather_dedup_scratch_bytes reports (12 bytes per index plus a hash table of at
 * least 16 bytes per index, all rounded up), 16-byte aligned, overwritten;
 * scratch_bytes too small: IBP_ERR_ARG. n_idx up to 2^24 - 1 and n_rows below 2^40,
 * else IBP_ERR_UNSUPPORTED. Asynchronous on s: three launches (clear, a gather that
 * claims each row as it goes, copy) for rows of at most 32 blocks and 4 KiB, four (a
 * hash pass before the gather) for longer rows; allocates nothing. */
int ibp_gather_dedup_scratch_bytes(int64_t n_idx, int64_t row_elems, int dtype,
                                   uint32_t block_elems, size_t *bytes);
int ibp_decompress_gather_dedup(const void *slots, int64_t slot_bytes, int64_t n_rows,
                                int64_t row_elems, int dtype, uint32_t block_elems,
                                const uint32_t *d_row_bitmask, const ibp_meta *d_meta,
                                const int64_t *d_idx, int64_t n_idx, void *out, void *d_scratch,
                                size_t scratch_bytes, int32_t *d_status, ibp_stream_t s);

/* ibp_decompress_gather given also the per-row bit counts ibp_compress wrote
 * (d_row_bits, n_rows words, device memory). A row's stored length is then known
 * from device memory before its slot is read, so exactly its used prefix (rounded
 * up to 16 bytes) is staged, with no round trip through the slot's header: for
 * slots in host memory only the stored bytes cross the link. A bit count that
 * disagrees with the row's header is reported as IBP_ERR_CORRUPT. */
int ibp_decompress_gather_sized(const void *slots, int64_t slot_bytes, int64_t n_rows,
                                int64_t row_elems, int dtype, uint32_t block_elems,
                                const uint32_t *d_row_bitmask, const uint32_t *d_row_bits,
                                const ibp_meta *d_meta, const int64_t *d_idx, int64_t n_idx,
                                void *out, int32_t *d_status, ibp_stream_t s);

/* One gather of a batch: a store (slots, slot_bytes, n_rows, its bitmask and
 * metadata) and the indices to read from it into out, as in ibp_decompress_gather. */
typedef struct {
  const void *slots;              /* device or registered host memory, 16-byte aligned */
  int64_t slot_bytes;
  int64_t n_rows;
  const uint32_t *d_row_bitmask;  /* device */
  const ibp_meta *d_meta;         /* device */
  const int64_t *d_idx;           /* device */
  int64_t n_idx;
  void *out;                      /* device, n_idx x row_elems words, 16-byte aligned */
} ibp_gather_job;

/* Several decompress-gathers with one row geometry (row_elems, dtype, block_elems)
 * in one launch per 64 jobs: e.g. one lookup batch per embedding table of a model.
 * jobs: host array of n_jobs descriptions (read during the call; the structs need
 * not outlive it). Each job gets CTAs in proportion to its indices, so the fixed
 * cost of a launch is paid once for the batch. Per-job checks, results and device
 * errors are those of ibp_decompress_gather (*d_status is shared by all jobs). */
int ibp_decompress_gather_batched(const ibp_gather_job *jobs, int n_jobs, int64_t row_elems,
                                  int dtype, uint32_t block_elems, int32_t *d_status,
                                  ibp_stream_t s);

/* Decompress a contiguous range of rows in order: out[i] = row row_begin + i for
 * i < n_out (row_begin + n_out <= n_rows). The same as ibp_decompress_gather with
 * d_idx = row_begin, row_begin + 1, ..., without an index array: for streaming
 * whole tensors (a layer's weights, a sequence's K/V rows) out of a store. */
int ibp_decompress_range(const void *slots, int64_t slot_bytes, int64_t n_rows, int64_t row_elems,
                         int dtype, uint32_t block_elems, const uint32_t *d_row_bitmask,
                         const ibp_meta *d_meta, int64_t row_begin, int64_t n_out, void *out,
                         int32_t *d_status, ibp_stream_t s);

/* Per-position metadata (a variant of preprocessing: the "kilobyte-scale" metadata
 * reading of "Core algorithm"; the paper fixes no layout, this one is the
 * library's). Element position e of a row (0 <= e < row_elems) has its own
 * mask/bitval pair, d_pmask[e] / d_pbitval[e] (w-bit values in uint32 words,
 * device memory, row_elems entries each): the preprocessing rule of ibp_build_meta
 * applied to the sample made of element e of every row. A block matches when each
 * of its elements e satisfies (x & pmask[e]) == pbitval[e]; a matching element is
 * stored as a field of w - popcount(pmask[e]) bits (its non-invariant bits,
 * ascending). Participation bits, bit order, shorter last blocks and the store rule
 * are those of the shared-mask format. Rows of at most 16 KiB (else
 * IBP_ERR_UNSUPPORTED); the argument checks of the shared-mask calls apply.
 * ibp_meta_positions_scratch_bytes: device scratch of ibp_build_meta_positions (8
 * bytes per bit of a row). */
int ibp_meta_positions_scratch_bytes(int64_t row_elems, int dtype, size_t *bytes);

int ibp_build_meta_positions(const void *rows, int64_t n_rows, int64_t row_elems, int dtype,
                             double T, uint32_t block_elems, uint32_t *d_pmask,
                             uint32_t *d_pbitval, void *d_scratch, ibp_stream_t s);

/* Block-position metadata (the block-sized reading of the "kilobyte-scale" metadata
 * of "Core algorithm", preprocessing; the layout is the library's). Position q of a
 * block (0 <= q < block_elems) gets one mask/bitval pair: the preprocessing rule of
 * ibp_build_meta applied to the sample made of the element at position q of every
 * block of every row (a shorter last block adds only the positions it has, so the
 * sample of position q has n_rows * ceil((row_elems - q) / block_elems) elements).
 * The result is written row-sized, like ibp_build_meta_positions: d_pmask[e] and
 * d_pbitval[e] (row_elems entries each, device memory) hold the pair of position
 * e % block_elems, so ibp_compress_positions and ibp_decompress_gather_positions
 * take them as they are. Same arguments, limits, scratch
 * (ibp_meta_positions_scratch_bytes) and errors as ibp_build_meta_positions;
 * asynchronous on s. */
int ibp_build_meta_block_positions(const void *rows, int64_t n_rows, int64_t row_elems,
                                   int dtype, double T, uint32_t block_elems, uint32_t *d_pmask,
                                   uint32_t *d_pbitval, void *d_scratch, ibp_stream_t s);

/* ibp_compress with per-position metadata (no *d_meta; no device-detected errors). */
int ibp_compress_positions(const void *rows, int64_t n_rows, int64_t row_elems, int dtype,
                           uint32_t block_elems, const uint32_t *d_pmask,
                           const uint32_t *d_pbitval, void *slots, int64_t slot_bytes,
                           uint32_t *d_row_bitmask, uint32_t *d_row_bits, ibp_stream_t s);

/* ibp_decompress_gather with per-position metadata. Each requested row's slot is
 * staged whole (its raw-size prefix). */
int ibp_decompress_gather_positions(const void *slots, int64_t slot_bytes, int64_t n_rows,
                                    int64_t row_elems, int dtype, uint32_t block_elems,
                                    const uint32_t *d_row_bitmask, const uint32_t *d_pmask,
                                    const uint32_t *d_pbitval, const int64_t *d_idx,
                                    int64_t n_idx, void *out, int32_t *d_status,
                                    ibp_stream_t s);

/* Statistics of a store ("System integration": a fixed-size buffer per tensor of
 * which only the compressed part is used, and a GPU-resident bitmask of the
 * compressed tensors; the statistics say how much of the buffers is used).
 * Reduces the bitmask and the per-row bit counts written by ibp_compress
 * (d_row_bitmask: ceil(n_rows/32) words, d_row_bits: n_rows words, device memory;
 * both may be null when n_rows == 0) into
 *   n_rows, n_compressed (bitmask bits set), raw_bytes (n_rows * row bytes),
 *   stored_bytes (sum of 4*ceil(bits/32) over compressed rows plus the raw row
 *   bytes of the others), total_bits (sum of the per-row bit counts).
 * ibp_query writes them to *h_out (host memory of any kind) and synchronises s
 * before it returns, so it cannot be captured in a CUDA graph. Its kernel reduces
 * into a 40-byte array built into the library (the library allocates nothing);
 * calls in one process take a lock around the launch and the wait, so two calls
 * never share the array. Errors: null h_out, n_rows < 0, row_elems <= 0 or a
 * non-device bitmask/bit-count pointer: IBP_ERR_ARG; unknown dtype: IBP_ERR_DTYPE;
 * a failed launch, copy or synchronisation: IBP_ERR_CUDA (*h_out then unchanged).
 * ibp_query_async: the same reduction into *d_stats (device memory, 8-byte
 * aligned, overwritten), asynchronous on s, capturable; same argument errors. */
int ibp_query(const uint32_t *d_row_bitmask, const uint32_t *d_row_bits, int64_t n_rows,
              int64_t row_elems, int dtype, ibp_stats *h_out, ibp_stream_t s);
int ibp_query_async(const uint32_t *d_row_bitmask, const uint32_t *d_row_bits, int64_t n_rows,
                    int64_t row_elems, int dtype, ibp_stats *d_stats, ibp_stream_t s);

/* ---- 8-bit paged key/value cache ------------------------------------------------
 * A lossy companion of the codec for the K/V rows it stores ("System integration":
 * offloaded inference keeps the KV cache as rows of tokens; the cache below is the
 * library's, the paper has no counterpart): the rows of the tokens attention reads on
 * the GPU are held in 8 bits an element with one scale for each page and head.
 *
 * Layout. At most 65535 sequences and 4096 heads. K codes, V codes:
 * [n_pages][n_heads][page_tokens][head_dim] bytes, each (page, head) one contiguous tile;
 * scales: [n_pages][n_heads] floats. Token t of sequence b lies in slot t % page_tokens of
 * page d_table[b*table_stride + t / page_tokens]; its value is code * scale. page_tokens
 * is 16, 32, 64 or 128, head_dim 64 or 128 (else IBP_ERR_UNSUPPORTED). A sequence holds at most table_cols *
 * page_tokens tokens (its capacity, at most 2^30). A page that a call writes (append: those
 * from a sequence's length on; evict: dst's) is named by one entry in use alone; others may
 * be shared by sequences. Entries past a sequence's last page are never read.
 *
 * Quantisation of a page's tile whose largest finite magnitude is a: scale = a * (1 /
 * qmax) (qmax 127 for IBP_KV_INT8, 448 for IBP_KV_E4M3) held in [2^-100, 2^120], or 0
 * when a is 0; code = value * (1 / scale), rounded to nearest even and saturated to +-qmax. A
 * NaN becomes code 0, an infinity the largest code of its sign (0 where the scale is 0).
 * All of it is IEEE single precision, so equal inputs give equal codes. Append and evict write
 * finite codes and scales only; in a pool that a caller fills, held tokens have scales that are
 * finite and not negative, and no NaN codes (eviction follows the rule above for others too; in
 * attention a value that is NaN may reach rows that do not see its token).
 *
 * Device-detected errors of these calls: a page id outside [0, n_pages), a length
 * outside [0, capacity] (it is clamped) or offsets that do not rise within [0, n_rows]
 * record IBP_ERR_INDEX in *d_status; tokens of such a page are skipped (not written, not
 * attended, read as zeros). */
typedef enum { IBP_KV_INT8 = 0, IBP_KV_E4M3 = 1 } ibp_kv_code;

typedef struct {
  void *k_codes, *v_codes;   /* device, 16-byte aligned */
  float *k_scales, *v_scales; /* device */
  const int32_t *d_table;    /* device, [batch][table_stride], table_cols of each row used */
  const int32_t *d_lens;     /* device, [batch]: tokens held by each sequence */
  int64_t n_pages, table_stride;
  int32_t batch, table_cols, n_heads, page_tokens, head_dim;
  int32_t code;              /* ibp_kv_code */
} ibp_kv_cache;

/* New K and V rows of the sequences, one after another: row r of K starts at k +
 * r*k_row_stride elements, its head h k_head_stride elements further (strides whole
 * multiples of 16 bytes, the elements of a head contiguous). Sequence b owns rows
 * d_cu[b] .. d_cu[b+1] - 1; d_cu null: n_rows / batch rows each. */
typedef struct {
  const void *k, *v;         /* device, 16-byte aligned, IBP_FP32, IBP_FP16 or IBP_BF16 */
  const int32_t *d_cu;       /* device, [batch + 1], or null */
  int64_t n_rows;
  int64_t k_row_stride, k_head_stride, v_row_stride, v_head_stride;
  int32_t dtype;
} ibp_kv_rows;

/* Append: sequence b's rows become its tokens d_lens[b], d_lens[b] + 1, ... in the pages
 * its table names. A page that already holds tokens keeps its scale s unless the new
 * rows need a larger one s'; the codes there then become round(code * (s / s')). A page
 * whose first slot is written starts a new scale. d_new_lens (nullable, [batch], not
 * d_lens itself) receives the lengths after the call; d_lens is not changed. Rows past
 * the capacity are dropped with IBP_ERR_INDEX (with offsets that do not rise, d_new_lens
 * may be written in part only). Calling it again with the same lengths
 * and rows leaves the pages as they are. Asynchronous on s, one launch. */
int ibp_kv_append(const ibp_kv_cache *cache, const ibp_kv_rows *rows, int32_t *d_new_lens,
                  int32_t *d_status, ibp_stream_t s);

/* Rotation of positions: d_table[p][i] holds the cosine and sine of pair i at position p. Pair
 * i of a head's first dim elements is (i, i + dim/2), or (2i, 2i + 1) when interleaved is not
 * 0; the rest of the head stays as it is. dim is a multiple of 16 from 16 to head_dim. A row
 * has a position on each of `axes` (1 to 4) axes, d_positions [n_rows][axes]; null: its
 * token's place in the cache (d_lens[b] and on) on every axis, which is its number in the
 * sequence until ibp_kv_evict leaves fewer tokens than there were: pass positions from then on. Pair i goes by the position on axis[i]
 * (axis[0 .. dim/2 - 1] < axes), so any layout of time, height and width is a matter of
 * axis[]. A pair (x, y) becomes (x c - y s, y c + x s), every product and sum rounded to
 * single precision. A position outside [0, n_positions) is held within it, with
 * IBP_ERR_INDEX. */
typedef struct {
  const float *d_table;      /* device, 16-byte aligned, [n_positions][dim/2][2] */
  const int32_t *d_positions; /* device, or null */
  int64_t n_positions;       /* 1 to 2^30 */
  int32_t dim, axes, interleaved;
  uint8_t axis[64];
} ibp_kv_rotation;

/* Query rows that are rotated with the new rows: row r belongs to the token that row r of K
 * becomes. Same type as K; strides as in ibp_kv_query; out is q itself (with its strides) or
 * shares no element with it, and in both cases none with K and V (else IBP_ERR_ARG, also where
 * rows of another stride than theirs lie in the same stretch of memory). */
typedef struct {
  const void *q;             /* device, 16-byte aligned */
  void *out;                 /* device, 16-byte aligned */
  int64_t q_row_stride, q_head_stride, out_row_stride, out_head_stride;
  int32_t q_heads;           /* 1 to 65535 */
} ibp_kv_turned;

/* ibp_kv_append with the rotation applied to K on the way: keys are quantised from the
 * rotated values in single precision (a NaN or infinity follows the quantisation's rule
 * after the rotation), values as they are. queries (nullable): rotated too and rounded once
 * to their type, whether or not there was room for their tokens; rows that belong to no
 * sequence (before d_cu[0], at or past d_cu[batch]) are left as they are. Asynchronous on s,
 * one launch or two, capturable. */
int ibp_kv_append_rotated(const ibp_kv_cache *cache, const ibp_kv_rows *rows,
                          const ibp_kv_rotation *rotation, const ibp_kv_turned *queries,
                          int32_t *d_new_lens, int32_t *d_status, ibp_stream_t s);

/* Read back: token d_begin[b] + i (d_begin null: i) of every sequence b, i < n_out, as
 * values rounded once to dtype into k_out and v_out ([batch][n_out][n_heads][head_dim],
 * either may be null; 16-byte aligned device memory): rows the codec's calls take.
 * Tokens at or past the length (or before 0) are written as zeros. */
int ibp_kv_read(const ibp_kv_cache *cache, const int32_t *d_begin, int64_t n_out, void *k_out,
                void *v_out, int dtype, int32_t *d_status, ibp_stream_t s);

/* Query rows of the sequences and what attention writes for them. Sequence b owns rows
 * d_cu[b] .. d_cu[b+1] - 1 (d_cu null: max_q rows each, n_rows = batch * max_q), at most
 * max_q of them; with n of them, row i stands at position d_lens[b] - n + i (the rows'
 * own keys are in the cache already) and sees the tokens up to and including it.
 * q_heads is a multiple of n_heads; query heads g*q_heads/n_heads .. share K/V head g.
 * dtype IBP_FP16 or IBP_BF16 (of q and out). Strides in elements, whole multiples of
 * 16 bytes; those of out put no two heads over one another (IBP_ERR_ARG). max_q at most
 * 2^30 (IBP_ERR_ARG), n_rows * q_heads / n_heads too (IBP_ERR_UNSUPPORTED). */
typedef struct {
  const void *q;             /* device, 16-byte aligned */
  void *out;                 /* device, 16-byte aligned, rows and heads strided */
  float *d_lse;              /* nullable, [n_rows][q_heads]: log of the sum of exponentials */
  const int32_t *d_cu;       /* nullable */
  const float *d_weights_in; /* nullable, [batch][n_heads][weights_stride] */
  float *d_weights;          /* nullable, same shape; may be d_weights_in itself */
  int64_t n_rows, max_q, weights_stride;
  int64_t q_row_stride, q_head_stride, out_row_stride, out_head_stride;
  int32_t q_heads, dtype;
  float scale, decay;
} ibp_kv_query;

/* Attention over the cache: out = sum_t p_t v_t with p = softmax over the tokens a row
 * sees of scale * q . k_t, sums and statistics in single precision (the factors p_t of
 * the sum are rounded to fp16, and bf16 queries to fp16 times a power of two); a row that
 * sees nothing gives zeros and lse = -inf. d_weights (weights_stride >= the capacity): for
 * t < d_lens[b], weights[b][h][t] = decay * weights_in[b][h][t] (0 when that is null) + the
 * sum of p_t over the rows and query heads of (b, h), in a fixed order; entries at or past
 * the length are left alone. The largest count chooses the kernel for all sequences of a
 * call: one with hundreds of rows is better attended apart from decoding ones. d_scratch: the size
 * ibp_kv_attention_scratch_bytes gives for the same cache and query shapes (16-byte
 * aligned; smaller: IBP_ERR_ARG), overwritten. With weights it holds n_rows * q_heads *
 * capacity floats of scores, but at most 1 GiB of them (or one row of one sequence): a
 * call that needs more goes over its rows in slices, a pair of launches each, in a fixed
 * order. Asynchronous on s, capturable. */
int ibp_kv_attention_scratch_bytes(const ibp_kv_cache *cache, int64_t n_rows, int64_t max_q,
                                   int32_t q_heads, int with_weights, size_t *bytes);
int ibp_kv_attention(const ibp_kv_cache *cache, const ibp_kv_query *query, void *d_scratch,
                     size_t scratch_bytes, int32_t *d_status, ibp_stream_t s);

/* Bounds of pages, for selecting among them: d_bounds [n_pages][n_heads][2][head_dim] (16-byte
 * aligned) receives the least and the largest K code of each element over the tokens that a
 * page holds, in units of scale * qmax / 127: for IBP_KV_INT8 the codes (-127 for -128), for
 * IBP_KV_E4M3 code * 127 / 448 rounded down (least) and up (largest; a NaN counts as 448 of its
 * sign); whole numbers in [-127, 127]. Written for the pages of the tokens from d_begin[b] (null or negative: 0) to
 * the length of each sequence, after an append the pages that it touched when d_begin holds
 * the lengths before it; other pages' bounds are left alone. A page that several sequences name
 * must hold equally many tokens in each. Asynchronous on s, capturable. */
int ibp_kv_bounds(const ibp_kv_cache *cache, int8_t *d_bounds, const int32_t *d_begin,
                  int32_t *d_status, ibp_stream_t s);

/* Early starts: the first kernel of ibp_kv_select, ibp_kv_attention_selected and
 * ibp_kv_attention_shared is launched with programmatic stream serialization. Where the kernel
 * before it on s is one that lets its dependents launch early (griddepcontrol.launch_dependents,
 * cudaTriggerProgrammaticLaunchCompletion), it starts while that one runs and waits for its end
 * before it reads or writes anything. What the three calls read they read through the first-level
 * cache. So a kernel of the caller's that lets them start early must not write, in any block, a
 * 128-byte line of their inputs that another of its blocks reads, and must itself have waited for
 * the kernel before it. Kernels that do not ask for this, and all calls of this interface, may
 * stand before them as they are.
 *
 * Selection of pages: for every sequence b and K/V head h, d_columns[b][h][0 .. pages - 1]
 * receives columns of the page table in rising order, then -1: all that the sequence has
 * where these are no more than `pages`, otherwise column 0, those where its query rows stand
 * (positions d_lens[b] - n and on) and of the others those of the highest scores, among equal
 * ones (a NaN is the lowest) the lowest column first. None for a sequence without rows.
 * The score of a page for a query row whose largest magnitude is in [2^e, 2^(e+1)), e held in
 * [-100, 100]: with n_d = q_d 2^(6-e) rounded to nearest even and held in [-127, 127] (0 for a
 * NaN), the whole number s = sum_d max(n_d least_d, n_d largest_d) of the page's bounds, times
 * 2^(e-6); the largest over the sequence's rows and the query heads that share h counts, times
 * the page's K scale, rounded once to single precision. It is the same on every run. Since no
 * token of a page has a product with the rounded query above it, the page that holds the
 * best token is not passed over for one that cannot hold a better one.
 * Of `query`, q, d_cu, n_rows, max_q, q_row_stride, q_head_stride, q_heads and dtype count.
 * pages holds column 0 and the rows' own: at least (max_q - 1 + page_tokens - 1) /
 * page_tokens + 2 (IBP_ERR_ARG). d_scratch: what ibp_kv_select_scratch_bytes gives (16-byte
 * aligned), overwritten. Asynchronous on s, capturable, one launch or two. */
int ibp_kv_select_scratch_bytes(const ibp_kv_cache *cache, size_t *bytes);
int ibp_kv_select(const ibp_kv_cache *cache, const int8_t *d_bounds, const ibp_kv_query *query,
                  int64_t pages, int32_t *d_columns, void *d_scratch, size_t scratch_bytes,
                  int32_t *d_status, ibp_stream_t s);

/* Attention over the pages that d_columns ([batch][n_heads][pages], as ibp_kv_select writes it)
 * names, as ibp_kv_attention over the whole cache (without weights: IBP_ERR_ARG). A sequence
 * has the smaller of `pages` and its number of pages as entries; the last of them must be the
 * columns where its rows stand, in order, the others columns before those in any order (one that
 * is named twice counts twice). A different entry is an IBP_ERR_INDEX and its page is left out. d_scratch: the size
 * ibp_kv_attention_selected_scratch_bytes gives. Asynchronous on s, capturable. */
int ibp_kv_attention_selected_scratch_bytes(const ibp_kv_cache *cache, int64_t n_rows, int64_t max_q,
                                            int32_t q_heads, int64_t pages, size_t *bytes);
int ibp_kv_attention_selected(const ibp_kv_cache *cache, const ibp_kv_query *query,
                              const int32_t *d_columns, int64_t pages, void *d_scratch,
                              size_t scratch_bytes, int32_t *d_status, ibp_stream_t s);

/* Attention of a batch whose sequences share beginnings, as ibp_kv_attention (without
 * weights: IBP_ERR_ARG). Group g is the sequences d_groups[g] .. d_groups[g+1] - 1 (d_groups
 * [n_groups + 1] rising within [0, batch], else IBP_ERR_INDEX; sequences of no group share
 * nothing); their first d_prefix[g] tokens are the same, and for the whole pages of these
 * their tables name the same pages (those of its first sequence with rows are read; pages in
 * use may be named more than once in calls that only read). A prefix longer than a
 * sequence, or than what the first of its rows sees, counts as far as all rows of the group
 * see it. Each beginning is gone over once for all rows of its group, in slabs of 128
 * sequences (unless the tables can hold no more than 64 MB of codes, or a sequence has more
 * than 64 rows a K/V head: then the call is that of ibp_kv_attention, and groups and prefixes are
 * not looked at). Dividing takes 6 to 10 us more before it gains anything: for short sequences
 * pass tables (table_cols) no wider than they need, or call ibp_kv_attention. Give pieces of
 * prompts a call of their own: one sequence of many rows leaves all undivided. A member of a group
 * whose first row sees less than a page of the prefix leaves the group nothing to share: let it
 * stand outside. group_rows: the most
 * query rows that the sequences of one group have together; it chooses the kernel, no result
 * depends on its being right. d_scratch: the size
 * ibp_kv_attention_shared_scratch_bytes gives for the same cache, query shapes and groups.
 * Asynchronous on s, capturable. */
int ibp_kv_attention_shared_scratch_bytes(const ibp_kv_cache *cache, int64_t n_rows, int64_t max_q,
                                          int32_t q_heads, int64_t n_groups, int64_t group_rows,
                                          size_t *bytes);
int ibp_kv_attention_shared(const ibp_kv_cache *cache, const ibp_kv_query *query, const int32_t *d_groups,
                            const int32_t *d_prefix, int64_t n_groups, int64_t group_rows,
                            void *d_scratch, size_t scratch_bytes, int32_t *d_status, ibp_stream_t s);

/* Eviction by accumulated weight: of every sequence b and head h longer than budget,
 * keeps the last `recent` tokens and, of the others, the budget - recent with the
 * largest d_weights[b][h][t] (equal weights: the lowest t first; a NaN counts as the
 * lowest); a shorter sequence keeps all. The kept tokens, in their order, become tokens
 * 0, 1, ... of dst (same heads, page size, head size, code and batch; pages distinct
 * from the source's; capacity >= the smaller of budget and the source's): values
 * code * scale requantised page by page. dst->d_lens is not read. d_new_lens [batch]
 * receives min(length, budget); d_new_weights (nullable, [batch][n_heads]
 * [new_weights_stride], new_weights_stride >= budget, apart from d_weights) the kept
 * weights, then zeros; d_kept (nullable, [batch][n_heads][budget]) the kept tokens' old
 * positions, then -1.
 * 0 <= recent <= budget, budget >= 1. Asynchronous on s, two launches. */
int ibp_kv_evict_scratch_bytes(const ibp_kv_cache *cache, int64_t budget, size_t *bytes);
int ibp_kv_evict(const ibp_kv_cache *cache, const float *d_weights, int64_t weights_stride,
                 int64_t budget, int64_t recent, const ibp_kv_cache *dst, int32_t *d_new_lens,
                 float *d_new_weights, int64_t new_weights_stride, int32_t *d_kept,
                 void *d_scratch, size_t scratch_bytes, int32_t *d_status, ibp_stream_t s);

/* Measurement helper, not part of the codec: streams `bytes` (a multiple of 16)
 * from src (device or registered host memory) with 16-byte loads across the whole
 * GPU and writes one XOR checksum word to *d_sink, so a caller can time the plain
 * read bandwidth of the memory the codec reads zero-copy. */
int ibp_probe_read(const void *src, int64_t bytes, uint64_t *d_sink, ibp_stream_t s);

#ifdef __cplusplus
}
#endif
#endif
