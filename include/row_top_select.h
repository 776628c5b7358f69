/*
 * row_top_select -- batched per-row exact top-K selection over indexer logits,
 * and the one-round candidate merge of a token-sharded (DCP) indexer, for AMD
 * Instinct MI355X (gfx950).
 *
 * Sources: the three pages this library follows.
 *   [P1] vLLM pull request 65178 (rank-major DCP top-k merge): "Overview" and
 *        "Details" -- (score, global id) candidates all-gathered along dim 0
 *        into [W, R, K, 2] and selected in place.
 *   [P2] vLLM API page vllm.models.kimi_k3.nvidia.ops.dcp_topk_merge.kernels:
 *        module docstring (B' word and bit plane, exactness, saturation word),
 *        DCPTopkPackKernel, DCPTopkSelectKernel, DCPTopkRescueKernel,
 *        DCPTopkRescueWorkspace, _decode_key, _ord16, dcp_topk_pack_indices,
 *        dcp_topk_select, dcp_topk_merge_rows, _check_exact.
 *   [P3] vLLM pull request 57206, "Use DeepSelect for eligible sparse-indexer
 *        prefill chunks": "Purpose" (causal per-row end, KV from column 0,
 *        preallocated output) and "Test Plan" (short rows, -1 tails, strided
 *        output, untouched padding, graph replay after updating row ends).
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is a DEVICE pointer owned by the caller; the
 *     library never allocates, frees or retains memory and keeps no state,
 *     except the static device scratch of topk_rows_noalloc (one array per
 *     GPU, its address cached on the first call there).
 *   - Every call only validates its arguments on the host and enqueues work on
 *     `stream` (0 = the null stream); it never synchronises, so calls are
 *     stream-ordered and may be captured into a HIP graph.  Data the kernels
 *     read (row_ends included) is read on the device at execution time.
 *   - Errors are reported by the return value (rts_status) before anything is
 *     launched; a failed launch returns RTS_EHIP.  Data-dependent oddities
 *     (NaN, out-of-range local ids, duplicate candidates) are defined
 *     behaviour and never cause an out-of-bounds access.
 *   - Scores order as IEEE values, descending, with -0.0 below +0.0 (the
 *     order of the order-preserving key of [P2] _ord16); NaN is never a
 *     candidate; +inf and -inf are ordinary candidates.  Equal scores are
 *     resolved toward the lower id.
 */
#ifndef ROW_TOP_SELECT_H
#define ROW_TOP_SELECT_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    RTS_OK = 0,
    RTS_EINVAL = -1,       /* a null pointer, a negative size, a stride below its row, ... */
    RTS_EUNSUPPORTED = -2, /* valid request outside what this build implements (e.g. k > 2048) */
    RTS_EWORKSPACE = -3,   /* a workspace was given but is smaller than required */
    RTS_EHIP = -4          /* the HIP runtime rejected the launch */
} rts_status;

typedef enum {
    RTS_F32 = 0,  /* IEEE binary32 */
    RTS_BF16 = 1, /* bfloat16 bit patterns (uint16_t) */
    RTS_E4M3 = 2  /* 8-bit float e4m3 (no infinities; index queries and keys only) */
} rts_dtype;

/* Human-readable name of an rts_status value (static storage). */
const char* rts_status_string(int status);

/*
 * Bytes of device workspace that lets topk_rows split long rows of a small
 * batch over several workgroups (0 when no split is used for this shape).
 * Passing less than this (but not 0) to topk_rows is RTS_EWORKSPACE; passing
 * no workspace at all is allowed and runs every row in one workgroup.
 */
size_t topk_rows_workspace_size(int dtype, int64_t rows, int64_t cols, int32_t k);

/*
 * topk_rows -- exact top-k of every row ([P3] Purpose and Test Plan; selection
 * rule of [P2] module docstring and DCPTopkSelectKernel docstring).
 *
 * logits    [rows, ld_logits] row-major, dtype RTS_F32 (float) or RTS_BF16
 *           (uint16_t bits); only columns [0, cols) are ever read, and of row i
 *           only columns [0, e_i).  Must be aligned to its element size.
 * row_ends  int32 [rows] or NULL.  e_i = clamp(row_ends[i], 0, cols): the
 *           exclusive causal end of row i, the row starting at column 0.
 *           NULL means e_i = cols for every row.
 * k         1 <= k <= 2048.
 * out_idx   int32 [rows, ld_out], ld_out >= k.  Row i receives the column ids
 *           of its m_i = min(k, #non-NaN in [0, e_i)) best entries in
 *           (score desc, id asc) order, then -1 in columns [m_i, k).  Columns
 *           [k, ld_out) are never written.
 * workspace optional device scratch (see topk_rows_workspace_size), may be
 *           NULL with workspace_bytes == 0.
 * Errors: RTS_EINVAL (bad sizes/strides/pointers/dtype/alignment),
 *         RTS_EUNSUPPORTED (k > 2048, cols >= 2^31), RTS_EWORKSPACE, RTS_EHIP.
 */
/* `dtype` is a plain int holding an rts_dtype value (RTS_F32 or RTS_BF16), so
 * the symbol keeps one fixed C signature for foreign-function callers; any
 * other value is RTS_EINVAL. */
int topk_rows(const void* logits, int dtype, int64_t rows, int64_t cols, int64_t ld_logits,
              const int32_t* row_ends, int32_t k, int32_t* out_idx, int64_t ld_out,
              void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * topk_rows_noalloc -- topk_rows for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc.  Same arguments (minus the workspace), outputs and
 * errors as topk_rows, and the same result.
 *
 * Where topk_rows would split long rows of a small batch over several
 * workgroups with a caller workspace, this call keeps the partial lists in a
 * static device array of the library instead: 16 MiB (every launch plan of
 * this library fits in it), one per GPU, held from the first call on that
 * GPU until the process ends.  The array's address on the current device is
 * taken on the first call there (make that first call outside graph
 * capture); no call allocates or frees memory.  Nothing in the array needs
 * clearing between calls: each launch writes every list it reads.  Calls on
 * one GPU share its array, so two calls whose executions overlap on that GPU
 * (different streams without ordering between them) race; calls ordered on
 * one stream do not.  A plan that needed more than the array holds would be
 * refused with RTS_EWORKSPACE.  `stream` must belong to the current device.
 */
int topk_rows_noalloc(const void* logits, int dtype, int64_t rows, int64_t cols, int64_t ld_logits,
                      const int32_t* row_ends, int32_t k, int32_t* out_idx, int64_t ld_out,
                      hipStream_t stream);

/*
 * pack_candidates -- a rank's local top-n as B' words ([P2] module docstring
 * step 1, DCPTopkPackKernel, dcp_topk_pack_indices).
 *
 * logits_bf16 [rows, ld_logits] bf16 bits; cols columns.
 * local_idx   int32 [rows, ld_idx], ld_idx >= n: local column ids, -1 padded,
 *             any order.
 * n           number of slots, a positive multiple of 32.
 * row_ends    int32 [rows] or NULL (= cols).
 * packed      int32 [rows, n + n/32], contiguous.  For slot j with
 *             l = local_idx[t, j] and end = min(row_end_t, cols, 2^17):
 *               0 <= l < end and score not NaN:
 *                 packed[t, j] = (ord16(score) << 16) | (0xFFFF - (l & 0xFFFF)),
 *                 bit j%32 of packed[t, n + j/32] = bit 16 of l;
 *               otherwise packed[t, j] = 0 (empty) and the plane bit is 0.
 *             ord16(b) = b & 0x8000 ? ~b & 0xFFFF : b | 0x8000.
 * Errors: RTS_EINVAL, RTS_EHIP.
 */
int pack_candidates(const uint16_t* logits_bf16, int64_t rows, int64_t cols, int64_t ld_logits,
                    const int32_t* local_idx, int32_t n, int64_t ld_idx, const int32_t* row_ends,
                    int32_t* packed, hipStream_t stream);

/*
 * merge_select_rank_major -- round-1 select of the packed merge ([P2] module
 * docstring steps 2-3 and saturation, DCPTopkSelectKernel, _decode_key; the
 * gathered buffer is read in place, rank-major, as in [P1]).
 *
 * gathered  int32 [world, rows, n + n/32], contiguous: rank r's packed rows.
 *           A nonzero word w at (r, t, j) is the candidate
 *             local = (0xFFFF - (w & 0xFFFF)) | (bit j%32 of gathered[r, t, n + j/32]) << 16,
 *             gid = local * world + r, score key ord16 = w >> 16.
 * world     1..16 ranks; n a positive multiple of 32; world * n <= 32768.
 * k         1 <= k <= 2048.
 * out_ids   int32 [rows, k], contiguous: the gids of the first min(k, count)
 *           candidates under (ord16 desc, gid asc), listed in candidate order
 *           (rank, then slot), then -1.
 * sat_word  int32 [rows] or NULL: (mask << 16) | tau16, tau16 = ord16 of the
 *           k-th selected (0 when fewer than k candidates), mask bit r set iff
 *           all n words of rank r are nonzero with ord16 > tau16; a mask with
 *           more than (k - 1) / n bits is cleared.  mask == 0 means round 1 is
 *           exact.
 * Candidates are expected to have distinct gids; with repeated words the
 * output stays in bounds and deterministic but is not specified further.
 * Limits are wider than the kernels page's (which takes k in {512, 1024,
 * 2048} and n < k without its second-round state): any k in [1, 2048] and
 * any n, since sat_word tells the caller whether round 1 was exact.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED, RTS_EHIP.
 */
int merge_select_rank_major(const int32_t* gathered, int32_t world, int64_t rows, int32_t n,
                            int32_t k, int32_t* out_ids, int32_t* sat_word, hipStream_t stream);

/*
 * merge_select_row_major -- merge_select_rank_major on the row-major layout
 * gathered int32 [rows, world, n + n/32] (rank r's words of row t at
 * gathered[t, r]), the layout an all-gather along dim 1 (or a reorder copy of
 * the dim-0 result) produces ([P1] Overview, "Before").  Same arguments,
 * limits, candidate order, outputs and errors; for the same words the outputs
 * are identical to merge_select_rank_major's.
 */
int merge_select_row_major(const int32_t* gathered, int32_t world, int64_t rows, int32_t n, int32_t k,
                           int32_t* out_ids, int32_t* sat_word, hipStream_t stream);

/*
 * Second round of the packed merge, with the world ranks on one device
 * ([P2] module docstring on exactness, DCPTopkRescueKernel,
 * DCPTopkRescueWorkspace).  A row enters it iff its sat_word mask is nonzero,
 * names only ranks below world and has at most S = (k - 1) / n bits (round 1
 * writes no other nonzero mask); every other row is neither read past its
 * sat_word nor written.  When S == 0 (n >= k) no row can enter and both calls
 * return RTS_OK without launching.  The receive buffer
 *   recv  int32 [rows, S, k + k/32], contiguous
 * holds, in slot s of row t, the packed local top-k of the s-th saturated
 * rank (ascending rank order), in the word and plane format of
 * pack_candidates with n = k.
 *
 * rescue_push -- rank `rank`'s push: for every row whose mask enters the
 * second round and has bit `rank`, copy local_packed[t] (int32 [rows,
 * k + k/32], contiguous: that rank's pack_candidates of its local top-k) into
 * recv[t, popc(mask & ((1 << rank) - 1))].  Other slots are not written.
 * 0 <= rank < world <= 16; n, k positive multiples of 32, k <= 2048.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED, RTS_EHIP.
 */
int rescue_push(const int32_t* local_packed, int32_t rank, int32_t world, int64_t rows, int32_t n,
                int32_t k, const int32_t* sat_word, int32_t* recv, hipStream_t stream);

/*
 * merge_rescue_rank_major -- the rescue select.  For every row that enters
 * the second round the candidates are, at flat position r * n + j, the
 * round-1 words gathered[r, t, j] (layout of merge_select_rank_major) of the
 * ranks whose bit is clear and whose ord16 >= tau16 (sat_word & 0xFFFF), then
 * at world * n + s * k + j the words of recv[t, s] for s < popc(mask), owned
 * by the s-th set bit.  out_ids[t] (int32 [rows, k], contiguous) is
 * overwritten with the gids of the first min(k, count) under (ord16 desc,
 * gid asc), in flat position order, then -1.  With the pushes of a valid
 * round 1 the selected scores equal the top-k of the union as a multiset.
 * world <= 16; n, k positive multiples of 32, k <= 2048;
 * world * n + min(S, world) * k <= 32768.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED, RTS_EHIP.
 */
int merge_rescue_rank_major(const int32_t* gathered, const int32_t* recv, int32_t world, int64_t rows,
                            int32_t n, int32_t k, const int32_t* sat_word, int32_t* out_ids,
                            hipStream_t stream);

/*
 * emit_rows -- this rank's owned physical KV rows of the selected ids ([P2]
 * DCPTopkSelectKernel docstring on emit_rows, dcp_topk_merge_rows: rows_out,
 * valid_out), the format sparse attention reads.
 *
 * ids         int32 [rows, k], contiguous: global ids as the selects write
 *             them (negative = empty slot).
 * world, dcp_rank  0 <= dcp_rank < world: a gid is owned iff
 *             gid % world == dcp_rank; its local index is gid / world.
 * req_id      int32 [rows]: the request (block-table row) of each row.
 * block_table int32 [table_rows, ld_table], first table_cols columns used:
 *             KV block ids of each request.
 * block_size  tokens per KV block (>= 1); stride_rows physical rows per block.
 * rows_out    int32 [rows, out_cols], contiguous, out_cols >= k: for each
 *             owned id, in the order ids lists them, the physical row
 *               block_table[req, b] * stride_rows + local % block_size,
 *             b = local / block_size (computed in 64 bits, stored as its low
 *             32 bits); then -1.  An id whose block b >= table_cols is
 *             dropped; a row whose req_id is outside [0, table_rows) owns
 *             nothing.
 * valid_out   int32 [rows]: the number of rows written for each row.
 * k <= 2048.  Errors: RTS_EINVAL, RTS_EUNSUPPORTED, RTS_EHIP.
 */
int emit_rows(const int32_t* ids, int64_t rows, int32_t k, int32_t world, int32_t dcp_rank,
              const int32_t* req_id, const int32_t* block_table, int64_t table_rows, int32_t table_cols,
              int64_t ld_table, int32_t block_size, int64_t stride_rows, int32_t* rows_out,
              int32_t out_cols, int32_t* valid_out, hipStream_t stream);

/*
 * rts_kv_rows -- where the fused selects below write this rank's owned
 * physical KV rows; the fields mean what the arguments of emit_rows of the
 * same names mean (all pointers device pointers, owned by the caller).
 */
typedef struct {
    int32_t dcp_rank;           /* 0 <= dcp_rank < world */
    const int32_t* req_id;      /* [rows] */
    const int32_t* block_table; /* [table_rows, ld_table], first table_cols columns used */
    int64_t table_rows;
    int32_t table_cols;
    int64_t ld_table;           /* >= table_cols */
    int32_t block_size;         /* >= 1 */
    int64_t stride_rows;
    int32_t* rows_out;          /* [rows, out_cols], contiguous, out_cols >= k */
    int32_t out_cols;
    int32_t* valid_out;         /* [rows] */
} rts_kv_rows;

/*
 * merge_select_rank_major_rows -- merge_select_rank_major that writes this
 * rank's owned physical rows straight from the select ([P2]
 * DCPTopkSelectKernel docstring: emit_ids and/or emit_rows;
 * dcp_topk_merge_rows).  For the same words, kv->rows_out and kv->valid_out
 * are exactly what emit_rows writes for the ids merge_select_rank_major
 * returns, and out_ids (optional, NULL = not written) and sat_word (NULL =
 * not written) are what merge_select_rank_major writes.
 * Errors: those of merge_select_rank_major; RTS_EINVAL for an invalid kv.
 */
int merge_select_rank_major_rows(const int32_t* gathered, int32_t world, int64_t rows, int32_t n,
                                 int32_t k, const rts_kv_rows* kv, int32_t* out_ids, int32_t* sat_word,
                                 hipStream_t stream);

/*
 * merge_rescue_rank_major_rows -- merge_rescue_rank_major that also (or
 * only: out_ids may be NULL) rewrites kv->rows_out and kv->valid_out of the
 * rows that enter the second round, as emit_rows would for their new ids.
 * Rows that do not enter are not written.
 * Errors: those of merge_rescue_rank_major; RTS_EINVAL for an invalid kv.
 */
int merge_rescue_rank_major_rows(const int32_t* gathered, const int32_t* recv, int32_t world,
                                 int64_t rows, int32_t n, int32_t k, const int32_t* sat_word,
                                 const rts_kv_rows* kv, int32_t* out_ids, hipStream_t stream);

/*
 * pack_pairs -- a rank's local top-kc as (score, global id) pairs ([P1]
 * Overview: "pack(local_topk)" into [R, K, 2]).
 *
 * logits    float [rows, ld_logits]; cols columns.
 * local_idx int32 [rows, ld_idx], ld_idx >= kc: local column ids, -1 padded.
 * row_ends  int32 [rows] or NULL (= cols).
 * rank, world  0 <= rank < world; cols * world < 2^31.
 * pairs     int32 [rows, kc, 2], contiguous: for l = local_idx[t, j] with
 *           0 <= l < clamp(row_end_t, 0, cols) and x[t, l] not NaN:
 *           (bits of x[t, l], l * world + rank); otherwise (0, -1).
 * Errors: RTS_EINVAL, RTS_EHIP.
 */
int pack_pairs(const float* logits, int64_t rows, int64_t cols, int64_t ld_logits,
               const int32_t* local_idx, int32_t kc, int64_t ld_idx, const int32_t* row_ends,
               int32_t rank, int32_t world, int32_t* pairs, hipStream_t stream);

/*
 * merge_select_pairs_rank_major -- select from (score, global id) pairs read
 * in place from the rank-major all-gather buffer ([P1] Overview and Details).
 *
 * gathered_pairs int32 [world, rows, kc, 2], contiguous: [..., 0] fp32 score
 *           bits, [..., 1] global id; a negative id is an empty slot, a NaN
 *           score is dropped.
 * world >= 1, kc >= 1, world * kc <= 32768.  k: 1 <= k <= 2048.
 * out_ids   int32 [rows, k], contiguous: the ids of the first min(k, count)
 *           candidates under (score desc, -0 below +0, id asc), listed in
 *           candidate order (rank, then slot), then -1.
 * Ids are expected to be distinct within a row (as all-gathered local top-k
 * lists are); repeated ids stay in bounds but are not specified further.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED, RTS_EHIP.
 */
int merge_select_pairs_rank_major(const int32_t* gathered_pairs, int32_t world, int64_t rows,
                                  int32_t kc, int32_t k, int32_t* out_ids, hipStream_t stream);

/*
 * merge_select_pairs_row_major -- merge_select_pairs_rank_major on the
 * row-major layout gathered_pairs int32 [rows, world * kc, 2] (candidate
 * r * kc + j of row t is rank r's slot j), the [R, W*K, 2] buffer of [P1]
 * Overview, "Before".  Same arguments, limits, order and errors; for the same
 * pairs the ids are identical to merge_select_pairs_rank_major's.
 */
int merge_select_pairs_row_major(const int32_t* gathered_pairs, int32_t world, int64_t rows,
                                 int32_t kc, int32_t k, int32_t* out_ids, hipStream_t stream);

/*
 * assign_slots -- places a batch's new tokens in a paged cache: block tables,
 * slot map and row ends from the requests' lengths, in the forms that
 * emit_rows (req_id, block_table), topk_rows (row_ends) and the calls below
 * read.
 *
 * ctx_lens   int32 [reqs]: tokens of each request already in the cache.
 * new_lens   int32 [reqs]: tokens that this step adds.  Negative lengths count
 *            as 0.  Token t of the batch belongs to the request i with
 *            query_starts[i] <= t < query_starts[i + 1].
 * reqs       0 <= reqs <= 8192.
 * tokens     capacity of the token outputs (a padded batch size); a request
 *            that reaches past it has its new tokens cut there.
 * block_size >= 1 tokens per block; stride_rows physical rows per block.
 * free_blocks int32 [free_count]: ids of free blocks, taken in order.
 * block_table int32 [reqs, ld_table], table_cols columns used, updated in
 *            place: request i keeps its first ceil(ctx / block_size) entries
 *            and gets the next free blocks in columns up to
 *            ceil((ctx + new) / block_size); requests take in ascending order.
 *            Where the list is exhausted the entry is -1; columns at or past
 *            table_cols are not written, though their blocks are taken.
 * query_starts int32 [reqs + 1]: exclusive sums of the (cut) new lengths.
 * req_id, row_ends, slots  int32 [tokens]: for token t of request i at
 *            position p = ctx + t - query_starts[i]: i, p + 1 and
 *            block_table[i, p / block_size] * stride_rows + p % block_size
 *            (its low 32 bits; -1 where the entry is negative or past the
 *            table).  Tokens behind the last request get -1, 0 and -1.
 * used       int32 [1]: blocks taken; more than free_count means that the
 *            list was too short.
 * No output may overlap an input or another output.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED (reqs > 8192, tokens or free_count >=
 *         2^31), RTS_EHIP.
 */
int assign_slots(const int32_t* ctx_lens, const int32_t* new_lens, int64_t reqs, int64_t tokens,
                 int32_t block_size, int64_t stride_rows, const int32_t* free_blocks,
                 int64_t free_count, int32_t* block_table, int32_t table_cols, int64_t ld_table,
                 int32_t* query_starts, int32_t* req_id, int32_t* row_ends, int32_t* slots,
                 int32_t* used, hipStream_t stream);

/*
 * indexer_logits -- the matrix that topk_rows selects from.  For query token t
 * and key s < e_t = clamp(row_ends[t], 0, cols):
 *   logits[t, s] = key_scales[s] * sum_h weights[t, h] * max(0, q[t, h, :] . keys[s, :])
 * with products and sums in 32 bits and one rounding at the end.  A NaN
 * product stays NaN.  Columns [e_t, ld_logits) are never written.
 *
 * q          [rows, heads, dim] of dtype RTS_BF16 or RTS_E4M3: row t at
 *            q + t * ld_q, its heads contiguous; ld_q in elements.
 * heads      1..128.  dim 64 or 128.
 * keys       [cols, dim], the same dtype, row stride ld_keys elements.
 * weights    float [rows, ld_weights], first heads columns (a query scale is
 *            the caller's to multiply in).
 * key_scales float [cols] or NULL (= 1).
 * row_ends   int32 [rows] or NULL (= cols).
 * logits     float or bf16 bits (logits_dtype RTS_F32 or RTS_BF16)
 *            [rows, ld_logits], ld_logits >= cols.
 * q and keys and their row strides must be multiples of 16 bytes.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED (dim, heads > 128, cols >= 2^31, ld_keys > 2^30),
 *         RTS_EHIP.
 */
int indexer_logits(const void* q, int dtype, int64_t rows, int32_t heads, int32_t dim, int64_t ld_q,
                   const void* keys, int64_t cols, int64_t ld_keys, const float* weights,
                   int64_t ld_weights, const float* key_scales, const int32_t* row_ends, void* logits,
                   int logits_dtype, int64_t ld_logits, hipStream_t stream);

/*
 * indexer_logits_paged -- indexer_logits with the keys of each token's request
 * read through its block table: column s of token t is the key at physical row
 *   block_table[req_id[t], s / block_size] * stride_rows + s % block_size
 * of key_cache [cache_rows, ld_keys] (key_scales [cache_rows] by the same row).
 * A key without a physical row (a negative block id, a row outside
 * [0, cache_rows), a block past table_cols) has the logit NaN, which topk_rows
 * drops; a token whose req_id is outside [0, table_rows) has no columns.
 * cols bounds every row end (ld_logits >= cols).  Neighbouring tokens of the
 * same request share the reads of their keys.
 * Errors: those of indexer_logits, RTS_EINVAL for block_size < 1, ld_table <
 *         table_cols, stride_rows < 0, RTS_EUNSUPPORTED for cache_rows >= 2^31.
 */
int indexer_logits_paged(const void* q, int dtype, int64_t rows, int32_t heads, int32_t dim,
                         int64_t ld_q, const void* key_cache, int64_t cache_rows, int64_t ld_keys,
                         const float* weights, int64_t ld_weights, const float* key_scales,
                         const int32_t* req_id, const int32_t* row_ends, const int32_t* block_table,
                         int64_t table_rows, int32_t table_cols, int64_t ld_table, int32_t block_size,
                         int64_t stride_rows, int64_t cols, void* logits, int logits_dtype,
                         int64_t ld_logits, hipStream_t stream);

/*
 * indexer_logits_plan -- how indexer_logits (table_rows -1) or
 * indexer_logits_paged would cut a call into workgroups, to read a profile or
 * to choose the sizes of a test by: plan[0] tokens a workgroup, plan[1] steps
 * of plan[2] columns each a workgroup, plan[3] stages of its rings of keys.
 * Host only; rows and cols at least 1.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED as those calls.
 */
int indexer_logits_plan(int dtype, int64_t rows, int32_t heads, int32_t dim, int64_t cols, int64_t table_rows,
                        int64_t* plan);

/*
 * latent_attend_rows -- attention over selected rows of a latent cache: one
 * vector c of d_latent + d_rope elements a cached token, shared by all heads,
 * is the key, and its first d_latent elements are the value (the queries come
 * with the key projection absorbed).  For row t and head h, over the entries
 * j < counts[t] with 0 <= ids[t, j] < cache_rows:
 *   z_j = scale * q[t, h, :] . cache[ids[t, j], :]
 *   lse[t, h] = log sum_j exp z_j,   out[t, h, :] = sum_j exp(z_j - lse) cache[ids[t, j], :d_latent]
 * Other entries (-1 tails among them) are not read and contribute nothing; a
 * row without entries gives zeros and -inf.  An id that occurs twice counts
 * twice.  A score of -inf has the weight 0 (and 0 times a value that is not
 * finite is NaN); where all are -inf, all weights are 0 and lse is -inf.
 * ids and counts are what emit_rows and the selects' rows forms write.
 *
 * q          bf16 [rows, heads, d_latent + d_rope]: row t, head h at
 *            q + t * ld_q + h * ld_head (elements).
 * scale      any number from -2^127 to 2^127.
 * d_latent   256 or 512; d_rope 64.
 * cache      bf16 [cache_rows, ld_cache].
 * ids        int32 [rows, ld_ids], first k columns used.
 * counts     int32 [rows] or NULL (= k); clamped to [0, k].
 * out        bf16 [rows, heads, d_latent], contiguous.
 * lse        float [rows, heads] or NULL.
 * workspace  optional device scratch, 16-byte aligned, of at least
 *            latent_attend_rows_workspace_size bytes: lets a small batch split
 *            each row's entries over several workgroups.  NULL with 0 bytes
 *            runs every row in one piece.  Calls in flight at the same time
 *            need workspaces of their own.
 * q, cache, out and their strides must be multiples of 16 bytes.
 * Scores, softmax statistics and sums are held in 32 bits; the weights are
 * rounded to bf16 for the products with the values.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED (d_latent, d_rope, heads > 1024,
 *         cache_rows >= 2^31),
 *         RTS_EWORKSPACE, RTS_EHIP.
 */
size_t latent_attend_rows_workspace_size(int64_t rows, int32_t heads, int32_t d_latent, int32_t k);
int latent_attend_rows(const void* q, int64_t rows, int32_t heads, int32_t d_latent, int32_t d_rope,
                       int64_t ld_q, int64_t ld_head, const void* cache, int64_t cache_rows,
                       int64_t ld_cache, const int32_t* ids, int32_t k, int64_t ld_ids,
                       const int32_t* counts, float scale, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

/*
 * latent_attend_paged -- latent attention of a batch's new tokens over their
 * requests' whole cache, read through the block table.  Request i has the new
 * tokens query_starts[i] .. query_starts[i + 1] and ctx_lens[i] cached tokens
 * before them; the new tokens' own vectors are already in the cache, at
 * positions ctx_lens[i] + j.  Token j of a request sees every position below
 * ctx_lens[i] and, of the new ones,
 *   tree == NULL: positions up to its own (causal);
 *   otherwise:    draft j' < 64 iff bit j' of tree[t] is set (a tree of drafted
 *                 tokens: the bits of its ancestors and its own).
 * Position p lies at physical row
 *   block_table[i, p / block_size] * stride_rows + p % block_size;
 * one without a physical row (as in indexer_logits_paged) is not seen.  What
 * is not seen never reaches a result, NaN and infinities included.  A token
 * that sees nothing gives zeros and -inf.  Rows of out and lse behind
 * query_starts[reqs] are not written.
 *
 * q, out, lse as in latent_attend_rows, over tokens rows (tokens bounds
 * query_starts).  query_starts int32 [reqs + 1], non-decreasing from 0.
 * tree       uint64 [tokens] or NULL.
 * ctx_lens   int32 [reqs], negative ones count as 0; positions from 2^31 - 64 on
 *            are not seen.
 * max_len    an upper bound of ctx_lens[i] + new tokens; it sets how the keys
 *            are split, results hold for any value >= 0.
 * workspace  as in latent_attend_rows, latent_attend_paged_workspace_size bytes.
 * Errors: as latent_attend_rows and indexer_logits_paged.
 */
size_t latent_attend_paged_workspace_size(int64_t tokens, int64_t reqs, int32_t heads,
                                          int32_t d_latent, int64_t max_len);
int latent_attend_paged(const void* q, int64_t tokens, int32_t heads, int32_t d_latent,
                        int32_t d_rope, int64_t ld_q, int64_t ld_head, const void* cache,
                        int64_t cache_rows, int64_t ld_cache, const int32_t* query_starts,
                        const int32_t* ctx_lens, int64_t reqs, const uint64_t* tree,
                        const int32_t* block_table, int32_t table_cols, int64_t ld_table,
                        int32_t block_size, int64_t stride_rows, int64_t max_len, float scale,
                        void* out, float* lse, void* workspace, size_t workspace_bytes,
                        hipStream_t stream);

/*
 * latent_attend_rows_plan, latent_attend_paged_plan -- how those calls would be
 * cut into workgroups, to read a profile or to choose the sizes of a test by:
 * plan[0] groups of 32 query rows a workgroup (1, 2 or 4), plan[1] pieces of a
 * row's keys at most.  split: whether the call has a workspace.  Host only;
 * rows and tokens and requests at least 1.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED as those calls.
 */
int latent_attend_rows_plan(int64_t rows, int32_t heads, int32_t d_latent, int32_t k, int split, int32_t* plan);
int latent_attend_paged_plan(int64_t tokens, int64_t reqs, int32_t heads, int32_t d_latent, int64_t max_len,
                             int split, int32_t* plan);

/*
 * merge_attend_rank_major -- joins the partial attentions of world ranks that
 * each own a part of the rows (emit_rows per dcp_rank, then
 * latent_attend_rows), read in place from the rank-major all-gather buffers:
 *   lse[t, h] = log sum_r exp lse_r[t, h],  out = sum_r exp(lse_r - lse) parts_r
 * A rank whose lse is -inf contributes nothing and its part is not read; if
 * all are, the result is zeros and -inf.
 *
 * parts      [world, rows, heads, dim] of dtype RTS_BF16 or RTS_F32, contiguous.
 * part_lse   float [world, rows, heads], contiguous.
 * world 1..64; dim a multiple of 8, at most 2048.
 * out        [rows, heads, dim] of out_dtype RTS_BF16 or RTS_F32, contiguous.
 * lse        float [rows, heads] or NULL.
 * parts and out must be 16-byte aligned.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED, RTS_EHIP.
 */
int merge_attend_rank_major(const void* parts, int dtype, const float* part_lse, int32_t world,
                            int64_t rows, int32_t heads, int32_t dim, void* out, int out_dtype,
                            float* lse, hipStream_t stream);

/*
 * beam_select -- beam search's selection over beams and vocabulary.  A group is
 * the beams of one request.  Beam b of group i has the score scores[i, b] and
 * the logits x of row i * beams + b; token v continues it with the value
 *   value(b, v) = scores[i, b] + x[v] - lse,   lse = log sum_v exp x[v]
 * and each group keeps the k best of all its beams' tokens.  Order: value
 * desc, then beam asc, then logit desc, token asc; within a beam it is that of
 * its logits, of which -0 and 0 are equal.
 * Values are formed in 64 bits and told apart to 2^-40 of
 * their size.  A row's sum has terms of 32 bits, so lse is off by up to
 * 2^-20 + 2^-23 of the mean (by weight) distance of the logits from their maximum,
 * some 1e-7 as a rule (for logits up to 1e6): beams whose values lie closer
 * than that may change places.  It is exact where one token has all of the
 * weight, and never below the largest logit: no value is above its beam's score.
 *
 * Not candidates: the token eos, tokens with a logit of -inf, beams whose score
 * is not finite (-inf marks a beam that is not in use, such as all but the
 * first at a search's first step) or whose logits hold a NaN, +inf or -inf only.
 *
 * logits     [groups * beams, ld_logits] of dtype RTS_F32 or RTS_BF16, vocab columns.
 * beams      1..64.   k  1..64.
 * scores     float [groups, beams].
 * eos        a token that ends a hypothesis, or -1 for none.
 * out_scores, parents, tokens  [groups, k], best first: the value (rounded to
 *            32 bits), the row i * beams + b of the beam and the token; then
 *            -inf, -1 and -1 where there are fewer candidates.  parents are
 *            what fork_blocks takes.
 * ended      float [groups, beams]: value(b, eos), -inf for beams that have no
 *            candidates.  NULL exactly where eos is -1.
 * workspace  device scratch, 16-byte aligned, of at least
 *            beam_select_workspace_size bytes; may be NULL where that is 0 (short rows of few
 *            beams).  Calls in flight at the same time need workspaces of their own.
 * out_scores may be scores where k is beams (refused otherwise); no other output may
 * overlap an input or another output.
 * Maxima and a sum's terms are held in 32 bits, sums over more than 32 terms and
 * values in 64.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED (beams, k, vocab >= 2^31, groups * beams
 *         >= 2^24), RTS_EWORKSPACE, RTS_EHIP.
 */
size_t beam_select_workspace_size(int dtype, int64_t groups, int32_t beams, int64_t vocab, int32_t k);
int beam_select(const void* logits, int dtype, int64_t groups, int32_t beams, int64_t vocab, int64_t ld_logits,
                const float* scores, int32_t k, int32_t eos, float* out_scores, int32_t* parents, int32_t* tokens,
                float* ended, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * fork_blocks -- the block table after rows were reordered, duplicated and
 * dropped: row i of the new table continues row parents[i] of the old one.
 * Rows share their parents' blocks; a block that more than one row would go on
 * writing into is given out anew, and is the caller's to copy (copy_blocks);
 * blocks that no row names any more are free.  Nothing is counted between
 * calls: which blocks are in use follows from the new rows and `held` alone.
 *
 * With len = max(0, ctx_lens[p]) of row i's parent p, the row has the parent's
 * first ceil(len / block_size) entries (of table_cols at most); the last of them
 * is being written if len is no multiple of block_size.  Row i keeps it if i is the first row of
 * p and the block is not held, not a whole block of any row and not
 * the last of another parent's rows; otherwise the r-th row that wants a
 * block of its own takes the r-th lowest free one and copies[r] = (the parent's
 * block, the new one).  Free are blocks that are neither held nor named by any
 * of these entries.  Where the pool is exhausted the entry is -1 and there is
 * no copy.  Other entries of the row are -1, as are entries outside [0, pool_blocks).
 *
 * block_table int32 [rows_in, ld_table], table_cols columns used.
 * ctx_lens   int32 [rows_in].
 * parents    int32 [rows_out]; outside [0, rows_in): an empty row, of length 0.
 *            A request ends when no row continues it.
 * pool_blocks blocks of the pool, at most 2^19; rows_in and rows_out at most 4096.
 * held       bytes [pool_blocks] or NULL: blocks that something else uses where
 *            not 0; they are never free and never kept for writing.
 * out_table  int32 [rows_out, ld_out]: table_cols columns are written.
 * out_lens   int32 [rows_out].
 * copies     int32 [rows_out, 2], 8-byte aligned, (-1, -1) behind the last; no
 *            block is both a source and a destination.
 * free_blocks int32 [n_free]: the ids that are free afterwards, ascending, then
 *            -1: a list for assign_slots.
 * counts     int32 [2]: how many are free afterwards (more than n_free, perhaps)
 *            and how many blocks the rows wanted (more than there are copies
 *            means that the pool was exhausted).
 * workspace  optional device scratch, 16-byte aligned, of at least
 *            fork_blocks_workspace_size bytes (0 where none is of use): lets several
 *            workgroups read a large table.  Calls in flight at the same time need
 *            workspaces of their own.
 * No output may overlap an input or another output (a table or lengths in place are
 * refused).
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED (rows, pool_blocks, table_cols >= 2^19),
 *         RTS_EWORKSPACE, RTS_EHIP.
 */
size_t fork_blocks_workspace_size(int64_t rows_in, int32_t table_cols, int32_t pool_blocks);
int fork_blocks(const int32_t* block_table, int64_t rows_in, int32_t table_cols, int64_t ld_table,
                const int32_t* ctx_lens, const int32_t* parents, int64_t rows_out, int32_t block_size,
                int32_t pool_blocks, const uint8_t* held, int32_t* out_table, int64_t ld_out, int32_t* out_lens,
                int32_t* copies, int32_t* free_blocks, int64_t n_free, int32_t* counts, void* workspace,
                size_t workspace_bytes, hipStream_t stream);

/*
 * compact_blocks -- moves that bring a pool's blocks in use to the lowest ids.
 * In use are the first ceil(ctx_lens / block_size) entries of each row; those that are
 * held stay where they are.  With n blocks in use that are not held, and T the
 * smallest bound below which n blocks are not held, the blocks in use at or past T move, in
 * ascending order, to the free ones below it.  A block that several rows share
 * moves once.  The caller copies the blocks (copy_blocks) before the new
 * table is used.
 *
 * max_moves  of the moves the first max_moves are made, the others left for
 *            another call.
 * out_table  int32 [rows, ld_out]: the table after the moves; entries past a
 *            row's length and outside [0, pool_blocks) become -1.
 * moves      int32 [max_moves, 2], 8-byte aligned: (from, to), then (-1, -1); no
 *            block is both.
 * free_blocks int32 [n_free]: the ids that are free after the moves, ascending, then -1.
 * counts     int32 [2]: how many are free, and how many moves there are in all.
 * Other arguments as in fork_blocks (rows * table_cols < 2^31), workspace with
 * compact_blocks_workspace_size bytes.
 * No output may overlap an input or another output (a table in place is refused).
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED, RTS_EWORKSPACE, RTS_EHIP.
 */
size_t compact_blocks_workspace_size(int64_t rows, int32_t table_cols, int32_t pool_blocks);
int compact_blocks(const int32_t* block_table, int64_t rows, int32_t table_cols, int64_t ld_table,
                   const int32_t* ctx_lens, int32_t block_size, int32_t pool_blocks, const uint8_t* held,
                   int32_t* out_table, int64_t ld_out, int32_t* moves, int64_t max_moves, int32_t* free_blocks,
                   int64_t n_free, int32_t* counts, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* A paged cache of any element type: rows of row_bytes bytes, ld_bytes apart. */
typedef struct {
    void* data;
    int64_t rows, row_bytes, ld_bytes;
} rts_cache;

/*
 * copy_blocks -- copies blocks within each of a number of caches (keys, values,
 * scales; the layers of a model): block b is the rows b * stride_rows .. +
 * block_size.
 *
 * caches     n_caches of them, at most 64; this array is on the HOST and is read
 *            before the call returns.
 * pairs      int32 [n_pairs, 2], 8-byte aligned: (from, to).  A pair with a
 *            negative id, of one block twice, or (in a cache) of a block that
 *            does not lie in it, is skipped.  No block may be the destination
 *            of two pairs, or of one and the source of another: what it then
 *            holds is not specified.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED (n_caches, rows, row_bytes or ld_bytes >=
 *         2^31), RTS_EHIP.
 */
int copy_blocks(const rts_cache* caches, int32_t n_caches, const int32_t* pairs, int64_t n_pairs, int32_t block_size,
                int64_t stride_rows, hipStream_t stream);

/*
 * kv_attend_paged -- attention of new tokens over their requests' paged cache of
 * keys and values.  The heads are in kv_heads groups of heads / kv_heads that
 * share a key head.  Token t sees the positions p < row_ends[t] of request
 * req_id[t] (its own is already in the cache) and, with a window, p >=
 * row_ends[t] - window, wherever the table ends.  For head h, of key head j, over what is seen:
 *   z_p = scale * k_scales[j] * q[t, h, :] . k[p, j, :],   lse[t, h] = log sum_p exp z_p
 *   out[t, h, :] = v_scales[j] * sum_p exp(z_p - lse) v[p, j, :]
 * Position p lies at physical row
 *   block_table[req_id[t], p / block_size] * stride_rows + p % block_size
 * of both caches; one without a physical row (as in indexer_logits_paged) is not
 * seen.  What is not seen never reaches a result, NaN and infinities included.
 * A token that sees nothing (a req_id outside [0, table_rows), such as a padded batch's,
 * among them) gives zeros and -inf.  A score of -inf has the weight 0 (and 0
 * times a value that is not finite is NaN); where all are -inf, all weights are 0 and lse is -inf.
 * req_id and row_ends are what assign_slots writes.
 *
 * q          bf16 [rows, heads, dim]: row t, head h at q + t * ld_q + h * ld_qhead (elements).
 * k_cache, v_cache  [cache_rows, kv_heads, dim] of dtype RTS_BF16 or RTS_E4M3: row r,
 *            head j at + r * ld_cache + j * ld_head (elements).
 * dim        64, 128 or 256.
 * k_scales, v_scales  float [kv_heads] or NULL (= 1).
 * window     positions seen at most, 0 for all.
 * max_len    an upper bound of row_ends; it says whether the keys are worth
 *            splitting, results hold for any value >= 0.
 * scale      any number from -2^127 to 2^127, and so its products with k_scales.
 * out        bf16 [rows, heads, dim], contiguous.   lse  float [rows, heads] or NULL.
 * workspace  as in latent_attend_rows, kv_attend_paged_workspace_size bytes.
 * q, the caches, out and their strides must be multiples of 16 bytes.
 * Scores, softmax statistics and sums are held in 32 bits; the weights enter the
 * products with the values as two bf16 terms (2^-16 of a weight is left out).
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED (dim, heads > 1024, rows * kv_heads *
 *         ceil(heads / kv_heads / 16) >= 2^25, rows * heads, cache_rows or
 *         table_rows >= 2^31, ld_cache > 2^30, ld_head > 2^40, a cache of 2^36
 *         bytes or more), RTS_EWORKSPACE, RTS_EHIP.
 */
size_t kv_attend_paged_workspace_size(int64_t rows, int32_t heads, int32_t kv_heads, int32_t dim, int dtype,
                                      int64_t max_len, int64_t window);
int kv_attend_paged(const void* q, int64_t rows, int32_t heads, int64_t ld_q, int64_t ld_qhead, const void* k_cache,
                    const void* v_cache, int dtype, int32_t kv_heads, int32_t dim, int64_t cache_rows,
                    int64_t ld_cache, int64_t ld_head, const float* k_scales, const float* v_scales,
                    const int32_t* req_id, const int32_t* row_ends, const int32_t* block_table, int64_t table_rows,
                    int32_t table_cols, int64_t ld_table, int32_t block_size, int64_t stride_rows, int64_t window,
                    int64_t max_len, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/*
 * kv_attend_paged_plan -- how that call would be cut, to read a profile or to choose
 * the sizes of a test by: plan[0] pieces that the rows' keys are cut into, about (0: a
 * row is one piece), plan[1] keys of a piece at least.  A call cuts all rows into
 * pieces of one size, by the lengths that it finds on the device.  split: whether
 * the call has a workspace.  Host only; rows at least 1.
 * Errors: RTS_EINVAL, RTS_EUNSUPPORTED as that call.
 */
int kv_attend_paged_plan(int64_t rows, int32_t heads, int32_t kv_heads, int32_t dim, int dtype, int64_t max_len,
                         int64_t window, int split, int64_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* ROW_TOP_SELECT_H */
