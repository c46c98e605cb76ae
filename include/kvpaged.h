/*
 * kvpaged.h -- C ABI of the GB300 paged KV-cache hot path (libkvpaged.so).
 *
 * Twenty-two calls, each one kernel launch on the caller's stream (the attentions
 * over the 4-bit cache and of drafted trees add a second one that joins the parts of
 * their split):
 *   kv_slot_mapping_paged    token -> cache slot through a block table
 *   kv_slot_mapping_paged_cp the same, for one rank of context parallelism
 *   kv_slot_mapping_range    token -> cache slot through contiguous ranges
 *   kv_cache_write           scatter new K/V rows into the paged caches
 *   kv_slot_mapping_paged_write  slot mapping and KV write in one launch
 *   kv_slot_mapping_range_write  the same through contiguous ranges
 *   kv_cache_gather          gather a request's K/V through its block table
 *   kv_cache_gather_bulk     the same gather, moved by bulk (TMA) copies
 *   kv_expand_kernel_blocks  manager-size block table -> kernel-size blocks
 *   kv_table_from_ranges     range descriptors -> block table
 *   kv_cache_gather_range    the gather, with blocks found from ranges
 *   kv_copy_blocks           copy-on-write copy of whole blocks
 *   kv_copy_blocks_bulk      the same copies, moved by bulk (TMA) copies
 *   kv_qk_norm_rope_write    per-head norm and rotation of q and k, K/V write
 *   kv_attention_prompt      causal attention of packed sequences
 *   kv_cache_write_q4        quantise new K/V rows into the 4-bit paged caches
 *   kv_cache_gather_q4       gather spans of the 4-bit caches as bf16 rows
 *   kv_attention_q4          one query token per request over the 4-bit caches
 *   kv_tree_layout           masks and positions of drafted trees from their parents
 *   kv_attention_tree        a step's rows (drafted trees, or one token) over the caches
 *   kv_verify_drafts         drafted tokens kept or refused, and one more token
 *   kv_cache_keep_path       the kept rows' K/V to consecutive positions, every layer
 *
 * Sources (page title, section):
 *   [BT]  "Blocktabelle" (vLLM v0.25.1 walkthrough)
 *   [VBM] "vLLM Block Table Management" (PagedAttention, vLLM V1 block stack)
 *   [RNG] "Range-addressed KV cache blocks for the vLLM serving engine"
 *
 * Common rules for every call
 * ---------------------------
 * Memory.  Every array argument is a device pointer owned by the caller
 *   (for example a torch CUDA tensor).  The library allocates nothing, keeps
 *   no state between calls and never synchronises: each call validates its
 *   host-visible arguments, enqueues one kernel on `stream` and returns.
 *   Kernels are launched with programmatic dependent launch: one may be
 *   scheduled while the previous kernel on the stream is finishing, but it
 *   waits for that kernel to complete before its first memory access, so the
 *   results are those of plain stream order (also inside CUDA graphs).
 *   A pointer may be NULL only where the call reads nothing through it (for
 *   example `positions` when num_tokens == 0).  What a call reads stays as it
 *   is until the call has ended: it may be read more than once, by blocks that
 *   rely on one another's findings.
 * Layouts.  All arrays are dense, row-major, without padding between rows
 *   other than the stated strides.  Block tables are int32
 *   [rows, table_stride]: row r is request r, column j the physical block of
 *   logical block j ([BT] Verantwortung).  Slot ids are int64, PAD = -1, and
 *   block 0 is the null block ([VBM] Symbol Map; Deep Dive 8).  K and V are
 *   separate bf16 caches [num_layers, num_blocks, block_size, num_kv_heads,
 *   head_dim]; the row of (layer, block, token) is
 *   n = (layer * num_blocks + block) * block_size + token and holds
 *   num_kv_heads * head_dim contiguous elements ([RNG] The Coordinate
 *   Approach).  All offsets are computed in 64 bits.
 * Status.  The return value is a kv_status: KV_OK, or a negative code when a
 *   host-visible argument is invalid (nothing is launched then), or
 *   KV_ECUDA when the launch itself failed.
 * Error word.  Data errors that only the device can see (a bad block id in a
 *   table, a slot outside the cache, a malformed range row ...) never fault
 *   and never stop the kernel: the affected token or row is skipped or
 *   padded as documented per call, and the matching KV_ERR_* bit is OR-ed
 *   into *d_err (int32, device memory, caller-cleared; d_err may be NULL to
 *   ignore such errors).  Read it after the stream has reached the call.
 * Empty work (zero tokens, zero requests) is valid and returns KV_OK.
 */
#ifndef KVPAGED_H
#define KVPAGED_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same underlying type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* kv_stream_t;

enum kv_status {
    KV_OK = 0,
    KV_EINVAL = -1,        /* null/misaligned pointer, negative or inconsistent size */
    KV_EUNSUPPORTED = -2,  /* a configuration the pages reject (fail closed) */
    KV_ECUDA = -3          /* the kernel launch failed */
};

enum kv_error_bits {
    KV_ERR_BAD_BLOCK = 1,     /* table/range block id outside [0, num_blocks) */
    KV_ERR_BAD_SLOT = 2,      /* write slot at or past num_blocks * block_size */
    KV_ERR_BAD_POSITION = 4,  /* negative position, or gather span invalid / past the table */
    KV_ERR_BAD_RANGE = 8,     /* descriptor count outside [0, range_stride] or a range length <= 0 */
    KV_ERR_NULL_WRITE = 16,   /* write slot inside the null block 0 */
    KV_ERR_BAD_QSL = 32,      /* query_start_loc decreasing, negative, or past num_tokens */
    KV_ERR_OUT_OF_SPACE = 64, /* gather rows exceed out_rows, or ranges exceed a table row */
    KV_ERR_TIMEOUT = 128,     /* an asynchronous bulk copy did not complete within the bounded
                                 wait (see "Bounded waits" below) */
    KV_ERR_BAD_TREE = 256,    /* a row's parent is no row before it, or a path does not go up */
    KV_ERR_BAD_TOKEN = 512,   /* drafted token outside [0, vocab) */
    KV_ERR_BAD_PROBS = 1024   /* no token has a probability above 0 */
};

/*
 * Bounded waits.  Only the two bulk-copy calls (kv_cache_gather_bulk,
 * kv_copy_blocks_bulk) wait on the copy engine, and kv_attention_prompt and
 * kv_attention_tree on it and on the matrix unit; every such wait gives up
 * after 1 s of GPU time (the global nanosecond timer) or 2^22 tries,
 * whichever comes first (kv_attention_prompt's counts from the fifth try; kv_attention_tree's
 * from the eighth, by the timer alone); a CTA that gave up waits once more, with the
 * bound of the bulk calls, for each of its own loads still in flight, then ends.  A healthy
 * copy completes in microseconds, so a timeout means the GPU is in trouble.
 * After a call has set KV_ERR_TIMEOUT:
 *   - its outputs are undefined: rows may be missing, partly written, or
 *     written after the kernel ended (a load still in flight when its CTA
 *     gave up), so do not use them;
 *   - treat later results on the same stream as suspect until the stream has
 *     been synchronised and checked for CUDA errors.
 * No wait in this library is unbounded.
 */

#define KV_PAD_SLOT_ID (-1)
#define KV_NULL_BLOCK_ID 0
#define KV_MAX_RANGES_PER_REQ 256   /* [RNG] The Fork Implementation: capped at 256 ranges */
#define KV_MAX_GATHER_REQS 4096     /* requests per kv_cache_gather(_range) call */
#define KV_MAX_TREE_ROWS 64         /* rows of a request's step: its last token and the drafted ones */
/* Largest max_num_tokens of one slot-mapping call (paged, range,
 * context-parallel, fused with the write): 2^31 - 65536, so that token indices
 * of a whole last tile stay in int32.  Larger values: KV_EINVAL. */
#define KV_MAX_TOKENS 2147418112

/*
 * kv_slot_mapping_paged -- per-token cache slot through the block table.
 *
 * Defined by [BT] Datenfluss (the slot-mapping kernel: block_index =
 * pos // block_size, block_number = block_table[req, block_index],
 * slot = block_number * block_size + pos % block_size; the last program pads
 * [num_tokens, max_num_tokens) with PAD) and [VBM] Deep Dive 8.
 *
 *   query_start_loc  int32 [num_reqs + 1]; request r owns tokens
 *                    [qsl[r], qsl[r+1]).  Must be non-decreasing.
 *   positions        int64 [num_tokens]; position of each token in its request.
 *   block_table      int32 [num_reqs, table_stride].
 *   slot_mapping     int64 [max_num_tokens], written entirely.
 *
 * For token t < num_tokens of request r with position p:
 *   p < 0                              -> PAD, KV_ERR_BAD_POSITION
 *   p / block_size >= table_stride     -> PAD
 *   b = block_table[r][p / block_size]:
 *     b == 0 (null block)              -> PAD  ([BT] CUDA-Graph-Padding: null rows are skipped)
 *     b < 0 or b >= num_blocks         -> PAD, KV_ERR_BAD_BLOCK
 *     otherwise                        -> b * block_size + p % block_size
 * Tokens in no request span, and tokens in [num_tokens, max_num_tokens), get
 * PAD.  A decreasing qsl, qsl[0] < 0 or qsl[num_reqs] > num_tokens sets
 * KV_ERR_BAD_QSL (slot values are then unspecified, but every store stays in
 * bounds).
 * Errors: KV_EINVAL for negative sizes, num_tokens > max_num_tokens,
 * max_num_tokens > KV_MAX_TOKENS, block_size <= 0, num_blocks < 1,
 * table_stride < 0, or a null/misaligned pointer that would be read.
 */
int kv_slot_mapping_paged(const int32_t* query_start_loc, const int64_t* positions,
                          const int32_t* block_table, int32_t table_stride, int32_t num_reqs,
                          int32_t num_tokens, int32_t max_num_tokens, int32_t block_size,
                          int64_t num_blocks, int64_t* slot_mapping, int32_t* d_err,
                          kv_stream_t stream);

/*
 * kv_slot_mapping_paged_cp -- kv_slot_mapping_paged filtered for one rank of
 * decode/prefill context parallelism.
 *
 * [BT] Entwurfsmotivation: with TOTAL_CP_WORLD_SIZE, TOTAL_CP_RANK and
 * CP_KV_CACHE_INTERLEAVE_SIZE the slot-mapping kernel writes real slots only
 * for the tokens of its own rank and PAD for all others; [VBM] Symbol Map:
 * DCP multiplies the block size of attention groups.  The pages stop before
 * the formula; this library's reading (its parity is pinned only at world
 * size 1 and by the partition properties): a table entry b names a virtual
 * block of block_size * W tokens, dealt to the W ranks in chunks of I tokens,
 * round robin; position p belongs to rank (p / I) % W and, on that rank, is
 * element ((p % (block_size*W)) / (I*W)) * I + p % I of physical block b, so
 * its slot is b * block_size + that element.  Each rank thus holds
 * block_size tokens of every virtual block, every token lives on exactly one
 * rank, and W = 1 gives kv_slot_mapping_paged.  All other rules (PAD, null
 * entries, errors, tail) are those of kv_slot_mapping_paged, with the table
 * indexed by p / (block_size * W).
 *
 *   cp_world_size W >= 1, 0 <= cp_rank < W, cp_interleave I >= 1.
 * Errors: as kv_slot_mapping_paged; KV_EINVAL for the ranges above or
 * block_size * W beyond int32; KV_EUNSUPPORTED when I does not divide
 * block_size.
 */
int kv_slot_mapping_paged_cp(const int32_t* query_start_loc, const int64_t* positions,
                             const int32_t* block_table, int32_t table_stride, int32_t num_reqs,
                             int32_t num_tokens, int32_t max_num_tokens, int32_t block_size,
                             int64_t num_blocks, int32_t cp_world_size, int32_t cp_rank,
                             int32_t cp_interleave, int64_t* slot_mapping, int32_t* d_err,
                             kv_stream_t stream);

/*
 * kv_slot_mapping_range -- per-token cache slot through contiguous ranges.
 *
 * Defined by [RNG] The Innovation: physical_block = range_start +
 * (pos // block_size - range_cum); positions outside every range get the
 * same PAD id as the paged call.  Descriptors are never loaded per position:
 * a lane reuses the range it resolved last, a warp of tokens of one request
 * reads 32 descriptors at once, and on large prefill batches a CTA stages
 * its tile's requests' first 32 descriptors in shared memory once.
 *
 *   range_start, range_len  int32 [num_reqs, range_stride]; request r's ranges
 *                           i < num_ranges[r] in logical order: range i holds
 *                           logical blocks [cum_i, cum_i + range_len[r][i])
 *                           with cum_i = sum of range_len[r][0..i-1], and
 *                           logical block cum_i + j is physical block
 *                           range_start[r][i] + j.
 *   num_ranges              int32 [num_reqs].
 *   other arguments         as kv_slot_mapping_paged.
 *
 * A logical block inside no range -> PAD.  The physical block b it resolves
 * to is checked like a table entry (0 -> PAD; outside [0, num_blocks) -> PAD
 * and KV_ERR_BAD_BLOCK).  A row with num_ranges[r] outside
 * [0, range_stride] sets KV_ERR_BAD_RANGE and all its tokens get PAD; a
 * range with length <= 0 sets KV_ERR_BAD_RANGE and covers no block.  Every
 * row r < num_reqs is validated, with or without tokens.
 * When block_table is the expansion of the ranges (and holds them all), the
 * two calls return identical slot_mapping and error words ([RNG] Benchmark
 * Methodology: both strategies produce identical slot ids).
 * Errors: as kv_slot_mapping_paged; range_stride > KV_MAX_RANGES_PER_REQ is
 * KV_EUNSUPPORTED ([RNG] The Fork Implementation: fail closed above 256).
 */
int kv_slot_mapping_range(const int32_t* query_start_loc, const int64_t* positions,
                          const int32_t* range_start, const int32_t* range_len,
                          const int32_t* num_ranges, int32_t range_stride, int32_t num_reqs,
                          int32_t num_tokens, int32_t max_num_tokens, int32_t block_size,
                          int64_t num_blocks, int64_t* slot_mapping, int32_t* d_err,
                          kv_stream_t stream);

/*
 * kv_cache_write -- scatter each new token's K and V rows to its slot.
 *
 * The cache write by slot of [BT] Verantwortung (kernels read and write KV
 * directly through slot_mapping) and [VBM] Deep Dive 8; multi-layer
 * addressing by [RNG] The Coordinate Approach.
 *
 *   key, value        bf16 [num_layers, num_tokens, num_kv_heads, head_dim].
 *   k_cache, v_cache  bf16 [num_layers, num_blocks, block_size, num_kv_heads, head_dim].
 *   slot_mapping      int64 [num_tokens].
 *
 * For every token t and layer l with s = slot_mapping[t]:
 *   s < 0 (PAD)                 -> skipped
 *   s / block_size == 0         -> skipped, KV_ERR_NULL_WRITE (block 0 is never written)
 *   s >= num_blocks*block_size  -> skipped, KV_ERR_BAD_SLOT
 *   otherwise cache row (l * num_blocks + s / block_size) * block_size + s % block_size
 *   of k_cache (v_cache) receives key[l][t] (value[l][t]) bit for bit.
 * Two tokens with the same slot race: each 16-byte piece of the row comes
 * from one of them, not necessarily the same one for every piece.
 * Errors: KV_EINVAL for a null or non-16-byte-aligned K/V pointer, negative
 * sizes, num_blocks < 1, block_size <= 0, num_kv_heads <= 0 or head_dim <= 0;
 * KV_EUNSUPPORTED when num_kv_heads * head_dim * 2 is not a multiple of 16.
 */
int kv_cache_write(const void* key, const void* value, void* k_cache, void* v_cache,
                   const int64_t* slot_mapping, int32_t num_tokens, int32_t num_layers,
                   int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                   int32_t head_dim, int32_t* d_err, kv_stream_t stream);

/*
 * kv_slot_mapping_paged_write -- kv_slot_mapping_paged, then kv_cache_write on
 * the slots it produced, in one launch.
 *
 * The slot of [BT] Datenfluss and the write by slot of [BT] Verantwortung
 * and [VBM] Deep Dive 8 with no trip through memory in between: each token's
 * K and V rows go straight to the slot computed for it.
 *
 *   query_start_loc .. num_blocks, slot_mapping  as kv_slot_mapping_paged;
 *                     slot_mapping is still written in full (PAD tail
 *                     included), for the attention kernels that read it.
 *   key, value        bf16 [num_layers, num_tokens, num_kv_heads, head_dim].
 *   k_cache, v_cache  bf16 [num_layers, num_blocks, block_size, num_kv_heads, head_dim].
 *
 * Results (slot_mapping, cache bytes, error bits) are exactly those of the
 * two calls in sequence; since a slot produced here is never in block 0 nor
 * past the pool, the write half adds no error bit of its own.  Tokens given
 * the same slot (a table that repeats a block) race as in kv_cache_write.
 * Errors: the union of the two calls' argument checks.
 */
int kv_slot_mapping_paged_write(const int32_t* query_start_loc, const int64_t* positions,
                                const int32_t* block_table, int32_t table_stride,
                                int32_t num_reqs, int32_t num_tokens, int32_t max_num_tokens,
                                int32_t block_size, int64_t num_blocks, const void* key,
                                const void* value, void* k_cache, void* v_cache,
                                int32_t num_layers, int32_t num_kv_heads, int32_t head_dim,
                                int64_t* slot_mapping, int32_t* d_err, kv_stream_t stream);

/*
 * kv_slot_mapping_range_write -- kv_slot_mapping_range, then kv_cache_write on
 * the slots it produced, in one launch ([RNG] The Innovation for the block,
 * otherwise as kv_slot_mapping_paged_write).
 *
 *   range_start, range_len, num_ranges, range_stride  as kv_slot_mapping_range.
 *   other arguments   as kv_slot_mapping_paged_write.
 *
 * Results are exactly those of kv_slot_mapping_range followed by
 * kv_cache_write, including KV_ERR_BAD_RANGE for every malformed row
 * r < num_reqs.  Errors: as kv_slot_mapping_range and kv_cache_write.
 */
int kv_slot_mapping_range_write(const int32_t* query_start_loc, const int64_t* positions,
                                const int32_t* range_start, const int32_t* range_len,
                                const int32_t* num_ranges, int32_t range_stride,
                                int32_t num_reqs, int32_t num_tokens, int32_t max_num_tokens,
                                int32_t block_size, int64_t num_blocks, const void* key,
                                const void* value, void* k_cache, void* v_cache,
                                int32_t num_layers, int32_t num_kv_heads, int32_t head_dim,
                                int64_t* slot_mapping, int32_t* d_err, kv_stream_t stream);

/*
 * kv_cache_gather -- read each request's K/V through its block table into
 * contiguous buffers (the read-path resolution of [RNG] Block-table lookup
 * per position; [VBM] Deep Dive 7: the kernel reads block_table[row][col]).
 *
 *   k_cache, v_cache  bf16 caches as in kv_cache_write; `layer` selects the layer.
 *   block_table       int32 [num_reqs, table_stride].
 *   gather_start/end  int32 [num_reqs]; request r asks for positions [start, end).
 *   k_out, v_out      bf16 [out_rows, num_kv_heads, head_dim].
 *
 * Requests are packed in order: position p of request r goes to output row
 * o_r + (p - start_r), o_r = sum of the earlier requests' lengths.  Each row:
 *   table entry b = block_table[r][p / block_size]:
 *     p / block_size >= table_stride -> zero row, KV_ERR_BAD_POSITION
 *     b == 0 (null block)            -> zero row (padding and recycled blocks)
 *     b < 0 or b >= num_blocks       -> zero row, KV_ERR_BAD_BLOCK
 *     otherwise                      -> cache row (layer, b, p % block_size)
 * A request with start < 0 or end < start contributes no rows and sets
 * KV_ERR_BAD_POSITION.  Rows at or past out_rows are not written and set
 * KV_ERR_OUT_OF_SPACE.  Output rows past the total are left untouched.
 * Errors: KV_EINVAL as kv_cache_write, or layer outside [0, num_layers),
 * out_rows < 0; KV_EUNSUPPORTED for a row size not a multiple of 16 bytes or
 * num_reqs > KV_MAX_GATHER_REQS (split the batch).
 */
int kv_cache_gather(const void* k_cache, const void* v_cache, int32_t layer, int32_t num_layers,
                    int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                    int32_t head_dim, const int32_t* block_table, int32_t table_stride,
                    const int32_t* gather_start, const int32_t* gather_end, int32_t num_reqs,
                    void* k_out, void* v_out, int64_t out_rows, int32_t* d_err,
                    kv_stream_t stream);

/*
 * kv_cache_gather_bulk -- kv_cache_gather done by the bulk-copy engine.
 *
 * Same arguments, output, packing, zero-row rules and error bits as
 * kv_cache_gather.  The rows of one request inside one cache block are moved
 * as one asynchronous bulk copy (global -> shared -> global, cp.async.bulk,
 * at most 32 KiB per copy) issued by a single thread per CTA, two one-warp
 * CTAs per SM: the whole-block gather with TMA bulk copies.  It reaches the
 * same bandwidth as kv_cache_gather while occupying 64 threads per SM, which
 * leaves the SMs to concurrent kernels.  Every wait for a copy is bounded
 * (see "Bounded waits"): if one ever ran out, KV_ERR_TIMEOUT is set and the
 * call's outputs are undefined.
 * Errors: as kv_cache_gather; KV_EUNSUPPORTED for a row of more than 32 KiB
 * (num_kv_heads * head_dim * 2 > 32768) or num_reqs > 2048.
 */
int kv_cache_gather_bulk(const void* k_cache, const void* v_cache, int32_t layer,
                         int32_t num_layers, int64_t num_blocks, int32_t block_size,
                         int32_t num_kv_heads, int32_t head_dim, const int32_t* block_table,
                         int32_t table_stride, const int32_t* gather_start,
                         const int32_t* gather_end, int32_t num_reqs, void* k_out, void* v_out,
                         int64_t out_rows, int32_t* d_err, kv_stream_t stream);

/*
 * kv_expand_kernel_blocks -- unfold manager blocks into kernel blocks.
 *
 * [BT] Entwurfsmotivation (map_to_kernel_blocks unfolds one manager block
 * into blocks_per_kv_block kernel blocks, e.g. manager 32 over kernel 16)
 * and Grenzen und Fehler (a kernel block size that does not divide the
 * manager block size is rejected).  With k = mgr_block_size /
 * kernel_block_size, manager entry m at column c becomes kernel entries
 * m*k + j at columns c*k + j, j < k; the null block 0 stays null (k zeros).
 * Columns at or past mgr_stride * k are set to 0.  An entry m < 0, or one
 * whose last kernel block would overflow int32, gives k null entries and
 * KV_ERR_BAD_BLOCK.
 *
 *   mgr_table     int32 [num_reqs, mgr_stride].
 *   kernel_table  int32 [num_reqs, kernel_stride], written entirely.
 * Errors: KV_EUNSUPPORTED when mgr_block_size % kernel_block_size != 0;
 * KV_EINVAL for block sizes <= 0, negative sizes, kernel_stride <
 * mgr_stride * k, or null pointers with work to do.
 */
int kv_expand_kernel_blocks(const int32_t* mgr_table, int32_t num_reqs, int32_t mgr_stride,
                            int32_t mgr_block_size, int32_t kernel_block_size,
                            int32_t* kernel_table, int32_t kernel_stride, int32_t* d_err,
                            kv_stream_t stream);

/*
 * kv_table_from_ranges -- materialise a block table from range descriptors.
 *
 * "Range-addressed KV cache blocks ...", Status: in range mode the staged
 * block table is copied to the kernels' table every step although the range
 * tables already hold the layout; a range-expansion kernel fills the table
 * directly.  Row r gets, in logical order, the blocks of request r's ranges:
 * logical block cum_i + j is range_start[r][i] + j (The Innovation).
 *
 *   range_start, range_len, num_ranges, range_stride  as kv_slot_mapping_range.
 *   block_table  int32 [num_reqs, table_stride], written entirely.
 *
 * Columns past the ranges are the null block 0.  A row with num_ranges[r]
 * outside [0, range_stride] is all null with KV_ERR_BAD_RANGE; a range with
 * length <= 0 covers nothing and sets KV_ERR_BAD_RANGE; ranges reaching past
 * table_stride are cut there with KV_ERR_OUT_OF_SPACE; an entry outside the
 * int32 range is null with KV_ERR_BAD_BLOCK.  kv_slot_mapping_paged on the
 * result equals kv_slot_mapping_range on the descriptors whenever no range is
 * cut.
 * Errors: KV_EINVAL for negative sizes or null/misaligned pointers with work
 * to do; KV_EUNSUPPORTED for range_stride > KV_MAX_RANGES_PER_REQ.
 */
int kv_table_from_ranges(const int32_t* range_start, const int32_t* range_len,
                         const int32_t* num_ranges, int32_t range_stride, int32_t num_reqs,
                         int32_t* block_table, int32_t table_stride, int32_t* d_err,
                         kv_stream_t stream);

/*
 * kv_cache_gather_range -- kv_cache_gather with the blocks found from range
 * descriptors instead of a block table (range arithmetic on the read path:
 * "Range-addressed KV cache blocks ...", The Direction, milestone M7, and the
 * planned comparison of the table gather against sequential range access in
 * Status).
 *
 * Arguments as kv_cache_gather, with (range_start, range_len, num_ranges,
 * range_stride) as in kv_slot_mapping_range in place of the table.  Output
 * rows, packing, spans, out_rows and the zero-row rules are those of
 * kv_cache_gather, where "table entry" reads "the block range arithmetic
 * gives": a logical block no range covers is a zero row (no error, like a
 * null entry); every row r < num_reqs with a malformed descriptor row sets
 * KV_ERR_BAD_RANGE and yields zero rows.  Equal to kv_cache_gather on the
 * table kv_table_from_ranges builds whenever every requested position lies
 * inside that table's stride.
 * Errors: as kv_cache_gather; range_stride > KV_MAX_RANGES_PER_REQ is
 * KV_EUNSUPPORTED.
 */
int kv_cache_gather_range(const void* k_cache, const void* v_cache, int32_t layer,
                          int32_t num_layers, int64_t num_blocks, int32_t block_size,
                          int32_t num_kv_heads, int32_t head_dim, const int32_t* range_start,
                          const int32_t* range_len, const int32_t* num_ranges,
                          int32_t range_stride, const int32_t* gather_start,
                          const int32_t* gather_end, int32_t num_reqs, void* k_out, void* v_out,
                          int64_t out_rows, int32_t* d_err, kv_stream_t stream);

/*
 * kv_copy_blocks -- batched whole-block copy for copy-on-write ("vLLM Block
 * Table Management", Deep Dive 3: KVCacheBlockCopy(src, dst) is queued so the
 * worker copies the KV data of a shared block into a fresh one before the
 * writer overwrites it).
 *
 *   k_cache, v_cache  bf16 [num_layers, num_blocks, block_size, kv_heads, head_dim],
 *                     read and written in place.
 *   src_blocks, dst_blocks  int32 [num_pairs].
 *
 * For every pair i and layer l, block dst_blocks[i] of K and of V becomes a
 * bit copy of block src_blocks[i].  A source outside [1, num_blocks) is
 * skipped with KV_ERR_BAD_BLOCK (block 0 holds no data); a destination 0 is
 * skipped with KV_ERR_NULL_WRITE; a destination outside [0, num_blocks) is
 * skipped with KV_ERR_BAD_BLOCK.  Destinations must be distinct and no
 * destination may be the source of another pair (as for freshly allocated
 * copy targets); otherwise copies race.  num_layers == 0 reads, writes and
 * checks nothing.
 * Errors: KV_EINVAL as kv_cache_write; KV_EUNSUPPORTED for a row size not a
 * multiple of 16 bytes.
 */
int kv_copy_blocks(void* k_cache, void* v_cache, int32_t num_layers, int64_t num_blocks,
                   int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                   const int32_t* src_blocks, const int32_t* dst_blocks, int32_t num_pairs,
                   int32_t* d_err, kv_stream_t stream);

/*
 * kv_copy_blocks_bulk -- kv_copy_blocks moved by the bulk-copy (TMA) engine.
 *
 * The same arguments, results, error bits and rules as kv_copy_blocks.  Each
 * K or V block of a (pair, layer) -- or each 32 KiB piece of a larger block --
 * goes global -> shared -> global with cp.async.bulk from one thread per
 * one-warp CTA, two CTAs per SM.  Every wait on the copy engine is bounded
 * (see "Bounded waits"): one that runs out sets KV_ERR_TIMEOUT, the kernel
 * ends normally, and the destination blocks are undefined.
 * Errors: as kv_copy_blocks; KV_ECUDA if the shared-memory size cannot be set.
 */
int kv_copy_blocks_bulk(void* k_cache, void* v_cache, int32_t num_layers, int64_t num_blocks,
                        int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                        const int32_t* src_blocks, const int32_t* dst_blocks,
                        int32_t num_pairs, int32_t* d_err, kv_stream_t stream);

/*
 * kv_qk_norm_rope_write -- what a layer does between its projection and its
 * attention: RMS norm of every query and key head, rotation by the token's
 * position, and the write of the new K and V rows to their slots.
 *
 *   query          bf16 [num_tokens, num_q_heads, head_dim]; key, value bf16
 *                  [num_tokens, num_kv_heads, head_dim].  The heads of a token
 *                  are dense; tokens are *_stride elements apart (the three may
 *                  be slices of one projection's output).
 *   q_weight, k_weight  bf16 [head_dim], the norms' weights.
 *   positions      int64 [num_tokens]; cos_sin fp32 [max_position, rotary_dim]:
 *                  rotary_dim/2 cosines, then as many sines, of a position's angles.
 *   q_out, k_out   bf16 [num_tokens, num_q_heads / num_kv_heads, head_dim], dense.
 *                  q_out may be query, and k_out key, where those rows are dense;
 *                  any other overlap with an input is refused.  k_out may be NULL
 *                  when there are caches.
 *   k_cache, v_cache, layer, num_layers, num_blocks, block_size, slot_mapping
 *                  as kv_cache_write, but only `layer` is written.  Both caches
 *                  NULL: no write, and value and slot_mapping are not read.
 *
 * For a head x: y = x * weight / sqrt(mean(x^2) + eps); then for i <
 * rotary_dim/2 with (a, b) = (y[i], y[i + rotary_dim/2]), or (y[2i], y[2i+1])
 * when `interleaved`: a' = a cos_i - b sin_i, b' = b cos_i + a sin_i.  Channels
 * at or past rotary_dim keep y.  All of it in 32 bits, rounded once.  V rows
 * are copied bit for bit.
 * A position outside [0, max_position) sets KV_ERR_BAD_POSITION: the token's
 * q_out and k_out rows are zero and nothing is cached.  Slots follow
 * kv_cache_write (PAD skipped; KV_ERR_NULL_WRITE; KV_ERR_BAD_SLOT); the outputs
 * are written in each of these cases.
 * Errors: KV_EINVAL for null or misaligned pointers (16 bytes; positions and
 * slots 8), sizes out of range, a stride below the row, rotary_dim outside
 * (0, head_dim], an overlap as above; KV_EUNSUPPORTED for head_dim above 256,
 * head_dim or rotary_dim not a multiple of 8, a stride not a multiple of 8, more than
 * 65535 query or KV heads, and more heads of all tokens together than a grid of
 * 2^31 - 1 CTAs holds (a CTA takes 4 warps, a warp 16 heads of up to 64 channels, 8 of
 * up to 128 or 4 of one token and kind).
 */
int kv_qk_norm_rope_write(const void* query, int64_t query_stride, const void* key,
                          int64_t key_stride, const void* value, int64_t value_stride,
                          const void* q_weight, const void* k_weight, const int64_t* positions,
                          const float* cos_sin, int64_t max_position, int32_t rotary_dim,
                          int32_t interleaved, float eps, int32_t num_tokens,
                          int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                          void* q_out, void* k_out, void* k_cache, void* v_cache, int32_t layer,
                          int32_t num_layers, int64_t num_blocks, int32_t block_size,
                          const int64_t* slot_mapping, int32_t* d_err, kv_stream_t stream);

/*
 * kv_attention_prompt -- causal attention of packed sequences with grouped
 * heads, over packed K/V rows: a prompt's own, or those kv_cache_gather(_q4)
 * read for a chunk behind earlier tokens.
 *
 *   query          bf16 [num_q_tokens, num_q_heads, head_dim]; key, value bf16
 *                  [num_k_tokens, num_kv_heads, head_dim]; strides as in
 *                  kv_qk_norm_rope_write.  Query head h reads KV head
 *                  h / (num_q_heads / num_kv_heads).
 *   q_start_loc, k_start_loc  int32 [num_reqs + 1]: request r owns query rows
 *                  [q_start_loc[r], q_start_loc[r+1]) and key rows
 *                  [k_start_loc[r], k_start_loc[r+1]).
 *   out            bf16 [num_q_tokens, num_q_heads, head_dim], dense, apart from
 *                  the inputs.
 *
 * With m query and n key rows, query i sees the keys j <= i + n - m:
 *   out_i = sum_j softmax_j(scale * q_i . k_j) v_j.
 * A query that sees no key gets zeros, as does one whose logits are all -infinity.  Keys a query does not see contribute
 * nothing to it, whatever they hold.  A NaN or an infinity in a value row makes
 * that channel NaN or infinite for the queries that see the row.  Query rows of
 * no request are left as they were.  A request whose rows are out of order or
 * out of range, or that has more than 2^24 key rows, sets KV_ERR_BAD_QSL and is
 * skipped; query rows that two requests claim (with such a one between them) hold
 * either's result, and where the requests claim more than num_q_tokens rows
 * together, some are left as they were.  Products and sums are held in 32 bits;
 * the weights are rounded to bf16 for their product with V.  Every wait of the
 * kernel is bounded (see "Bounded waits").
 * Errors: KV_EINVAL for null or misaligned pointers, negative sizes, a stride
 * below the row, num_q_heads not a multiple of num_kv_heads, a scale that is
 * not positive and finite, out overlapping an input; KV_EUNSUPPORTED for head_dim
 * above 128 or not a multiple of 8, a stride not a multiple of 8, more than 128
 * query heads per KV head, num_q_heads > 4096, num_reqs > KV_MAX_GATHER_REQS, more
 * than KV_MAX_TOKENS query or key rows, and where the sequences' tile pairs (of 256 / group
 * tokens, group being the query heads per KV head, rounded down) times num_kv_heads may be more
 * than 2^31 - 1.
 */
int kv_attention_prompt(const void* query, int64_t query_stride, const void* key,
                        int64_t key_stride, const void* value, int64_t value_stride,
                        const int32_t* q_start_loc, const int32_t* k_start_loc,
                        int32_t num_reqs, int32_t num_q_tokens, int32_t num_k_tokens,
                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                        void* out, int32_t* d_err, kv_stream_t stream);

/*
 * The 4-bit paged cache.  K and V are separate byte arrays [num_layers,
 * num_blocks, num_kv_heads, record], a record being block_size *
 * (head_dim/2 + head_dim/16) bytes: the block's tokens' codes (head_dim/2 bytes
 * each), then their scales (one bf16 per 32 channels).  With G = head_dim/32,
 * byte 2 G g + 2 j + b (g < 8, j < G, b < 2) of a token's codes holds channel
 * 32 j + 4 g + 2 b in its low four bits and the next channel in its high ones;
 * a code c stands for (c - 8) * scale of its group j of 32 channels.
 * head_dim is 64 or 128 and block_size a multiple of 8 (else KV_EUNSUPPORTED;
 * also above 4096 KV heads).  Whole blocks are copied by kv_copy_blocks with
 * block_size = num_kv_heads, num_kv_heads = 1 and head_dim = record / 2.
 *
 * kv_cache_write_q4 -- kv_cache_write into `layer` of the 4-bit caches.
 *
 *   key, value    bf16 [num_tokens, num_kv_heads, head_dim], strides as in
 *                 kv_qk_norm_rope_write.
 *   slot_mapping  int64 [num_tokens], rules and error bits of kv_cache_write.
 *
 * Per group of 32 channels x: scale = bf16(max|x| / 7), code = round(x / scale)
 * + 8, nearest with ties to even.  A scale below 2^-126 makes the group zeros; a
 * group with a NaN or an infinity gets a NaN scale and reads as NaN.  Two tokens
 * with the same slot race: the row is then undefined.  KV_EUNSUPPORTED also where
 * num_tokens * num_kv_heads passes 16 * (2^31 - 1).
 */
int kv_cache_write_q4(const void* key, int64_t key_stride, const void* value,
                      int64_t value_stride, void* k_cache, void* v_cache,
                      const int64_t* slot_mapping, int32_t num_tokens, int32_t layer,
                      int32_t num_layers, int64_t num_blocks, int32_t block_size,
                      int32_t num_kv_heads, int32_t head_dim, int32_t* d_err,
                      kv_stream_t stream);

/*
 * kv_cache_gather_q4 -- kv_cache_gather from the 4-bit caches: bf16 rows
 * [out_rows, num_kv_heads, head_dim] of the values the codes stand for (rounded
 * to bf16).  Packing, spans, zero rows, out_rows and error bits are those of
 * kv_cache_gather.
 */
int kv_cache_gather_q4(const void* k_cache, const void* v_cache, int32_t layer,
                       int32_t num_layers, int64_t num_blocks, int32_t block_size,
                       int32_t num_kv_heads, int32_t head_dim, const int32_t* block_table,
                       int32_t table_stride, const int32_t* gather_start,
                       const int32_t* gather_end, int32_t num_reqs, void* k_out, void* v_out,
                       int64_t out_rows, int32_t* d_err, kv_stream_t stream);

/*
 * kv_attention_q4 -- attention of one query token per request over the 4-bit
 * caches (a decode step).
 *
 *   query          bf16 [num_reqs, num_q_heads, head_dim], tokens query_stride
 *                  elements apart; query head h reads KV head
 *                  h / (num_q_heads / num_kv_heads).
 *   block_table    int32 [num_reqs, table_stride].
 *   span_start, span_end  int32 [num_reqs]: request r attends its positions
 *                  [start, end) (a sliding window starts late).
 *   out            bf16 [num_reqs, num_q_heads, head_dim], dense, apart from the inputs.
 *   workspace      device memory, 16-byte aligned, of at least
 *                  kv_attention_q4_workspace() bytes on the same device; it
 *                  holds no state between calls, and two calls that may run at
 *                  the same time need one each.
 *
 *   out = sum_p softmax_p(scale * q . k_p) v_p
 * over the positions whose table entry is a block of the pool.  Null entries are
 * left out; entries outside [0, num_blocks) are left out with KV_ERR_BAD_BLOCK,
 * positions past the table row with KV_ERR_BAD_POSITION.  A request with no
 * position left, or with start < 0 or end < start (KV_ERR_BAD_POSITION), gets
 * zeros.
 * Products and sums are held in 32 bits; a weight times a value scale is rounded to
 * fp16 for its product with the codes: by 2^-11 of it at most, or, where it lies more
 * than 2^21 below the largest of its query and channel group, by 2^-32 of that one
 * (or by 2^-133, where those are near the end of the 32-bit range).
 * Queries of 2^100 and more and value scales above 2^100 may give infinities or
 * NaN.  The same call gives the same bits every time.
 * Errors: as kv_attention_prompt and the 4-bit cache; KV_EINVAL for a workspace
 * that is missing, misaligned, too small or shared with out or an input; KV_EUNSUPPORTED for a layer of more
 * than 2^36 bytes in one cache.
 */
int kv_attention_q4(const void* query, int64_t query_stride, const void* k_cache,
                    const void* v_cache, int32_t layer, int32_t num_layers, int64_t num_blocks,
                    int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                    int32_t head_dim, const int32_t* block_table, int32_t table_stride,
                    const int32_t* span_start, const int32_t* span_end, int32_t num_reqs,
                    float scale, void* out, void* workspace, int64_t workspace_bytes,
                    int32_t* d_err, kv_stream_t stream);

/* Workspace bytes of a kv_attention_q4 call on the current device (0 for none), or
 * KV_EINVAL for sizes out of range. */
int64_t kv_attention_q4_workspace(int32_t num_reqs, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim);

/*
 * Drafted trees.  A step of a request has m rows (1 .. KV_MAX_TREE_ROWS): row 0 is its last
 * token, whose K and V are not cached yet, every other row a drafted token that follows its
 * parent, a row before it.  Rows of all requests are packed: request r owns rows
 * [q_start_loc[r], q_start_loc[r+1]) of num_rows.  With n = context_len[r] tokens cached, row
 * i's K and V go to cache position n + i, whatever its place in the tree; its rotation is by
 * position n + depth.  A step: kv_tree_layout; in every layer kv_qk_norm_rope_write (slots
 * by kv_slot_mapping_paged of the cache positions) and kv_attention_tree; kv_verify_drafts;
 * kv_cache_keep_path.  A request whose rows are out of order, out of range or too many
 * sets KV_ERR_BAD_QSL and is skipped: its rows of the outputs are left as they were, as
 * are rows of no request (rows that two requests claim, with such a one between them, hold
 * either's).  All four calls: at most KV_MAX_GATHER_REQS requests and
 * KV_MAX_TREE_ROWS * KV_MAX_GATHER_REQS rows (else KV_EUNSUPPORTED).
 *
 * kv_tree_layout -- what each row sees and where it stands.
 *
 *   parents          int32 [num_rows]: the index, in its request, of each row's parent
 *                    (row 0's is not read); NULL: chains, the parent is the row before.
 *   q_start_loc      int32 [num_reqs + 1]; context_len int32 [num_reqs].
 *   tree_mask        int64 [num_rows]: bit j of row i: row j is row i or above it.
 *   positions        int64 [num_rows]: context_len + depth (0 for row 0).
 *   cache_positions  int64 [num_rows]: context_len + i.
 *
 * A row whose parent is not a row before it sets KV_ERR_BAD_TREE and stands like row 0: it
 * sees itself, at depth 0.  A negative context_len sets KV_ERR_BAD_POSITION where its request
 * has rows; both positions of those are -1.
 * Errors: KV_EINVAL for negative counts, null or misaligned pointers (tree_mask and
 * positions 8 bytes, others 4), an output that shares bytes with an input or another output.
 */
int kv_tree_layout(const int32_t* parents, const int32_t* q_start_loc, const int32_t* context_len,
                   int32_t num_reqs, int32_t num_rows, int64_t* tree_mask, int64_t* positions,
                   int64_t* cache_positions, int32_t* d_err, kv_stream_t stream);

/*
 * kv_attention_tree -- attention of a step's rows over the bf16 paged caches; with one row
 * a request, a decode step.
 *
 *   query          bf16 [num_rows, num_q_heads, head_dim], rows query_stride elements
 *                  apart; query head h reads KV head h / (num_q_heads / num_kv_heads).
 *   k_cache, v_cache, layer, ..  as kv_cache_write; `layer` is read.
 *   block_table    int32 [num_reqs, table_stride].
 *   q_start_loc    int32 [num_reqs + 1].
 *   span_start     int32 [num_reqs]: first visible position of the context (a sliding
 *                  window starts late); NULL: 0.
 *   context_len    int32 [num_reqs].
 *   tree_mask      int64 [num_rows]: row i sees row j of its request (position
 *                  context_len + j) where bit j is set, itself included; bits at and past
 *                  the request's rows mean nothing.  NULL: row i sees the rows j <= i.
 *   max_rows       1 .. KV_MAX_TREE_ROWS: no request has more rows (KV_ERR_BAD_QSL).  Every request's
 *                  keys are read once for each 256 of max_rows * (num_q_heads / num_kv_heads), or
 *                  part of them, whatever rows it has: give no more than the batch has, and a few
 *                  requests of many rows a call of their own.
 *   out            bf16 [num_rows, num_q_heads, head_dim], dense, apart from the inputs.
 *   workspace      as kv_attention_q4, of kv_attention_tree_workspace() bytes.
 *
 *   out_i = sum_p softmax_p(scale * q_i . k_p) v_p
 * over the positions [span_start, context_len) and the rows row i sees, as far as their table
 * entry is a block of the pool.  Of the positions [span_start, context_len + rows), null entries
 * are left out, entries outside [0, num_blocks) are left out with KV_ERR_BAD_BLOCK, positions past
 * the table row with KV_ERR_BAD_POSITION.  A row with no position left, or whose logits are all -infinity, gets
 * zeros; so do the rows of a request with span_start < 0 or context_len < span_start
 * (KV_ERR_BAD_POSITION).  Positions a row does not see contribute nothing to it, whatever they hold.
 * A NaN or an infinity in a value row makes that channel NaN or infinite for the rows that
 * see it.  Products and sums are held in 32 bits; the weights are rounded to bf16 for
 * their product with V.  Logits (scale * q_i . k_p) of 2^30 and more may give NaN or zeros.  The same
 * call gives the same bits every time.
 * Errors: KV_EINVAL for null or misaligned pointers, sizes out of range, a stride below the
 * row, num_q_heads not a multiple of num_kv_heads, a scale that is not positive and finite, a
 * workspace that is missing, misaligned or too small, out or workspace sharing bytes with
 * each other or an input; KV_EUNSUPPORTED for head_dim above 128 or not a multiple of 8, a
 * stride not a multiple of 8, more than 64 query heads per KV head, num_q_heads > 4096, a pool of
 * more than 2^31 - 1 tokens (num_blocks * block_size).
 */
int kv_attention_tree(const void* query, int64_t query_stride, const void* k_cache,
                      const void* v_cache, int32_t layer, int32_t num_layers, int64_t num_blocks,
                      int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                      int32_t head_dim, const int32_t* block_table, int32_t table_stride,
                      const int32_t* q_start_loc, const int32_t* span_start,
                      const int32_t* context_len, const int64_t* tree_mask, int32_t num_reqs,
                      int32_t num_rows, int32_t max_rows, float scale, void* out, void* workspace,
                      int64_t workspace_bytes, int32_t* d_err, kv_stream_t stream);

/* Workspace bytes of a kv_attention_tree call on the current device (0 for none), or
 * KV_EINVAL / KV_EUNSUPPORTED for sizes out of range. */
int64_t kv_attention_tree_workspace(int32_t num_reqs, int32_t max_rows, int32_t num_q_heads,
                                    int32_t num_kv_heads, int32_t head_dim);

/*
 * kv_verify_drafts -- which drafted tokens are kept, and the token behind them.
 *
 *   target_probs  [num_rows, vocab], rows target_stride elements apart: the target's
 *                 probabilities of the token that follows each row.
 *   draft_probs   the same, rows draft_stride apart: the probabilities each row's children
 *                 were drawn from, independently; rows without children are not read.  NULL:
 *                 the drafted tokens were not drawn (the likeliest ones, a lookup).
 *   prob_type     KV_F32 or KV_BF16, of both.
 *   tokens        int32 [num_rows]: each row's token (row 0's is not read).
 *   parents       as kv_tree_layout.
 *   uniform       fp32 [num_rows], in [0, 1): row i's number decides on its token, row 0's draws
 *                 the last token.
 *   out_tokens    int32 [num_rows]: the kept tokens, then the last one, then -1.
 *   path          int32 [num_rows]: the kept rows from row 0 on, then -1.
 *   num_kept      int32 [num_reqs]: kept drafted tokens; num_kept + 1 entries of the other
 *                 two are not -1 (0 for a request that is skipped or has no rows).
 *
 * At row i (from row 0 on), with p and q its rows of the two, s_0 = p and Z_0 = 1, its
 * children are tried in order: child c with token x and number u is kept when
 *   u q(x) Z_j < s_j(x),   else   s_(j+1) = max(s_j - Z_j q, 0),  Z_(j+1) = sum s_(j+1).
 * Without draft_probs q is 1 at x and 0 elsewhere, and Z_(j+1) = Z_j - s_j(x).  A kept child is the next
 * row.  With no child left, the last token is the smallest t with sum_(k <= t) s(k) > u_0 sum_k
 * s(k); where s is 0 everywhere, s = p.  So the tokens are distributed as the target's.
 * Sums are held in integers of 2^-45 and 64 bits, whose order does not matter; a weight is
 * a multiple of 2^-45, off by less than that.  The same call gives the same bits every time.  (Rows that
 * sum to 2^18 and more are no probabilities: the last token is then any, or -1.)
 * Probabilities below 0 and NaN count as 0, above 1 as 1; numbers below 0 and NaN count as 0, of 1 and
 * above as the largest below 1.  A token outside [0, vocab) is passed over with
 * KV_ERR_BAD_TOKEN; so is a row whose parent is not a row before it (KV_ERR_BAD_TREE) and
 * those below it.  Where p is 0 everywhere the last token is -1 (KV_ERR_BAD_PROBS).
 * Errors: KV_EINVAL for negative counts, vocab < 1, a prob_type that is neither, a stride below
 * vocab, null pointers or pointers not aligned to their elements, an output that shares bytes with
 * an input or another output; KV_EUNSUPPORTED for vocab > 2^20.
 */
enum kv_prob_type { KV_F32 = 0, KV_BF16 = 1 };
int kv_verify_drafts(const void* target_probs, int64_t target_stride, const void* draft_probs,
                     int64_t draft_stride, int32_t prob_type, int32_t vocab, const int32_t* tokens,
                     const int32_t* parents, const int32_t* q_start_loc, const float* uniform,
                     int32_t num_reqs, int32_t num_rows, int32_t* out_tokens, int32_t* path,
                     int32_t* num_kept, int32_t* d_err, kv_stream_t stream);

/*
 * kv_cache_keep_path -- the kept rows' K and V to consecutive positions, in every layer of
 * the bf16 caches, in place: of request r, for i = 1 .. num_kept[r], the rows of cache
 * position context_len + path[i] go to position context_len + i.
 *
 *   k_cache, v_cache, ..  as kv_cache_write.
 *   block_table, context_len, q_start_loc  as kv_attention_tree.
 *   path, num_kept        as kv_verify_drafts: path goes up from 0.
 *
 * The rows behind the last kept one stay as they were, for the next step to overwrite.  Blocks that
 * requests share must not hold a moved position.  A request is left as it was where num_kept
 * is negative or not below its rows, or path does not start at 0 and go up inside them
 * (KV_ERR_BAD_TREE), context_len is negative or a position past the table row
 * (KV_ERR_BAD_POSITION), or a moved row's block, old or new, is the null block
 * (KV_ERR_NULL_WRITE) or outside the pool (KV_ERR_BAD_BLOCK).
 * Errors: KV_EINVAL for sizes out of range, null or misaligned pointers (caches 16 bytes), caches that
 * share bytes with each other or with another argument; KV_EUNSUPPORTED for a row
 * (num_kv_heads * head_dim) that is no multiple of 8.
 */
int kv_cache_keep_path(void* k_cache, void* v_cache, int32_t num_layers, int64_t num_blocks,
                       int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                       const int32_t* block_table, int32_t table_stride,
                       const int32_t* q_start_loc, const int32_t* context_len, const int32_t* path,
                       const int32_t* num_kept, int32_t num_reqs, int32_t num_rows, int32_t* d_err,
                       kv_stream_t stream);

/*
 * kv_diag_bounded_wait -- self-test of the bounded wait the bulk-copy gather
 * relies on.  No page defines it: it exists so the timeout path can be
 * exercised on a real GPU without faulting or hanging it.  One thread waits,
 * for at most spin_limit tries, on a shared-memory barrier that nothing will
 * complete; when the limit runs out it OR-s KV_ERR_TIMEOUT into *d_err and
 * the kernel ends normally, so the context stays usable.
 *   spin_limit  1 .. 2^20 tries.
 *   d_err       int32 device word (required).
 * Errors: KV_EINVAL for a limit out of range or a null/misaligned d_err.
 */
int kv_diag_bounded_wait(int32_t spin_limit, int32_t* d_err, kv_stream_t stream);

/*
 * kv_diag_role_wait -- the same for the wait that the roles of kv_attention_prompt share:
 * four warps wait, each on a shared-memory barrier that nothing will complete.  The last
 * one gives up after limit_ns; the others, whose own limit is 1 s, leave when it has.
 *   limit_ns     0 .. 10^9.
 *   d_waited_ns  int64 [4]: how long each warp waited.
 *   d_err        int32 device word (required): KV_ERR_TIMEOUT.
 * Errors: KV_EINVAL for a limit out of range or a null/misaligned pointer.
 */
int kv_diag_role_wait(int64_t limit_ns, int64_t* d_waited_ns, int32_t* d_err,
                      kv_stream_t stream);

/*
 * kv_diag_attention_prompt_stall -- self-test of kv_attention_prompt's bounded waits, through
 * its own kernels: in every CTA, as it starts on its work number `item` (counted from 0; a CTA
 * without that much work runs on as usual), one role waits limit_ns for a barrier that nothing
 * will complete, then gives up.  The CTA's other roles leave at their next wait, it waits for its
 * copies and matrix instructions in flight and ends; KV_ERR_TIMEOUT arrives; the context stays
 * usable.  The outputs are undefined.
 *   role      0 copies, 1 matrix instructions, 2 check of values, 3 and 4 softmax.
 *   limit_ns  0 .. 10^9.
 *   d_err     required.
 * Errors: those of kv_attention_prompt; KV_EINVAL for a role, item or limit out of range.
 */
int kv_diag_attention_prompt_stall(const void* query, int64_t query_stride, const void* key,
                                   int64_t key_stride, const void* value, int64_t value_stride,
                                   const int32_t* q_start_loc, const int32_t* k_start_loc,
                                   int32_t num_reqs, int32_t num_q_tokens, int32_t num_k_tokens,
                                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                   float scale, void* out, int32_t* d_err, int32_t role,
                                   int32_t item, int64_t limit_ns, kv_stream_t stream);

/* Human-readable name of a kv_status value (static string). */
const char* kv_status_string(int status);

/* ABI version of this header (bumped on any signature change; a call that is added leaves it). */
int kv_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KVPAGED_H */
