// Host-side launchers implemented next to their kernels and called by the
// C ABI in rts_api.cpp after argument validation.  Each returns an rts_status.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace rts {

// A rank's owned physical KV rows, emitted by a packed select next to (or
// instead of) the global ids (kernels page: DCPTopkSelectKernel docstring on
// emit_rows, dcp_topk_merge_rows).  rows_out == nullptr: not requested.
struct RowsArgs {
    const int32_t* req_id;       // [rows]
    const int32_t* block_table;  // [table_rows, ld_table]
    int32_t* rows_out;           // [rows, out_cols]
    int32_t* valid_out;          // [rows]
    int64_t table_rows, ld_table, stride_rows;
    int32_t dcp_rank, table_cols, block_size, out_cols;
};

// Launch geometry of topk_rows for one problem shape.
struct TopkPlan {
    int e;          // sorted-list length per lane (list = 64 * e >= k)
    int waves;      // waves per workgroup sharing one row
    int groups;     // workgroups per row (> 1 needs a workspace)
    size_t ws_bytes;
    int block_kpt;  // > 0: whole rows in one workgroup's registers, block_kpt keys per thread
};

// Largest workspace a topk_rows plan uses: partial lists of split rows beyond
// this take fewer groups.  Also the size of topk_rows_noalloc's static scratch.
constexpr size_t kMaxSplitBytes = size_t(16) << 20;

TopkPlan plan_topk_rows(int dtype, int64_t rows, int64_t cols, int32_t k, bool allow_split);

// topk_rows_noalloc's scratch on the current device (its address there, taken
// on the first call on the device) and its size in bytes.
int scratch_of_current_device(void** ptr, size_t* bytes);

int launch_topk_rows(const void* logits, int dtype, int64_t rows, int64_t cols, int64_t ld,
                     const int32_t* row_ends, int32_t k, int32_t* out, int64_t ld_out,
                     const TopkPlan& plan, void* workspace, hipStream_t stream);

int launch_pack_candidates(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                           const int32_t* local_idx, int32_t n, int64_t ld_idx,
                           const int32_t* row_ends, int32_t* packed, hipStream_t stream);

int launch_pack_pairs(const float* x, int64_t rows, int64_t cols, int64_t ld,
                      const int32_t* local_idx, int32_t kc, int64_t ld_idx,
                      const int32_t* row_ends, int32_t rank, int32_t world, int32_t* pairs,
                      hipStream_t stream);

// row_major: gathered is [rows, world, n + n/32] instead of [world, rows, n + n/32].
int launch_merge_packed(const int32_t* gathered, bool row_major, int32_t world, int64_t rows,
                        int32_t n, int32_t k, int32_t* out_ids, int32_t* sat_word,
                        const RowsArgs* rows_args, hipStream_t stream);

// Candidate slots of one rescued row: world * n round-1 words plus k words
// for each of at most min((k-1)/n, world) receive slots.
int rescue_candidates(int32_t world, int32_t n, int32_t k);

int launch_rescue_push(const int32_t* local_packed, int32_t rank, int32_t world, int64_t rows,
                       int32_t n, int32_t k, const int32_t* sat_word, int32_t* recv,
                       hipStream_t stream);

int launch_merge_rescue(const int32_t* gathered, const int32_t* recv, int32_t world, int64_t rows,
                        int32_t n, int32_t k, const int32_t* sat_word, int32_t* out_ids,
                        const RowsArgs* rows_args, hipStream_t stream);

int launch_emit_rows(const int32_t* ids, int64_t rows, int32_t k, int32_t world, int32_t dcp_rank,
                     const int32_t* req_id, const int32_t* block_table, int64_t table_rows,
                     int32_t table_cols, int64_t ld_table, int32_t block_size, int64_t stride_rows,
                     int32_t* rows_out, int32_t out_cols, int32_t* valid_out, hipStream_t stream);

// row_major: pairs is [rows, world * kc, 2] instead of [world, rows, kc, 2].
int launch_merge_pairs(const int32_t* pairs, bool row_major, int32_t world, int64_t rows,
                       int32_t kc, int32_t k, int32_t* out_ids, hipStream_t stream);

// ------------------------------------------------------------------ paged caches

// Requests' block tables over a cache of physical rows.
struct Pages {
    const int32_t* table;  // [table_rows, ld]
    int64_t table_rows, ld, stride_rows, cache_rows;
    int32_t cols, block_size;
    int32_t shift;  // log2(block_size), or -1 where it is no power of two
};

inline Pages make_pages(const int32_t* table, int64_t table_rows, int32_t cols, int64_t ld,
                        int32_t block_size, int64_t stride_rows, int64_t cache_rows) {
    int32_t shift = -1;
    for (int32_t i = 0; i < 31; ++i)
        if (block_size == (1 << i)) shift = i;
    // A cache has fewer than 2^31 rows: with a stride of 2^31 or more only block 0 has any, and the
    // products of block ids and such strides could pass 64 bits.
    if (stride_rows > (1ll << 31)) stride_rows = 1ll << 31;
    return Pages{table, table_rows, ld, stride_rows, cache_rows, cols, block_size, shift};
}

constexpr int64_t kMaxThreads = 0xFFFFFFFFll;  // of one launch, along x

constexpr int64_t kMaxReqs = 8192;  // assign_slots keeps two sums a request in LDS

int launch_assign_slots(const int32_t* ctx_lens, const int32_t* new_lens, int64_t reqs, int64_t tokens,
                        int32_t block_size, int64_t stride_rows, const int32_t* free_blocks,
                        int64_t free_count, int32_t* block_table, int32_t table_cols, int64_t ld_table,
                        int32_t* query_starts, int32_t* req_id, int32_t* row_ends, int32_t* slots,
                        int32_t* used, hipStream_t stream);

// The arguments of indexer_logits and indexer_logits_paged; req_id == nullptr:
// the keys are rows [0, cols) of `keys`, the same for every token.
struct LogitsArgs {
    const void *q, *keys;
    const float *weights, *key_scales;
    const int32_t *row_ends, *req_id;
    void* logits;
    int64_t rows, cols, ld_q, ld_keys, ld_weights, ld_logits;
    Pages pages;
    int32_t heads, dim;
    int dtype, logits_dtype;
};
int launch_indexer_logits(const LogitsArgs& a, hipStream_t stream);

// How a call is cut into workgroups.
struct LogitsPlan {
    int tokens;         // of a workgroup
    int stages;         // of its waves' rings of keys
    int step;           // columns that all its waves take at a time
    int64_t steps;      // of a workgroup
    int64_t lds;        // bytes
};
// `reqs`: requests of the paged form, or -1.
LogitsPlan plan_indexer_logits(int dtype, int64_t rows, int64_t cols, int32_t heads, int32_t dim, int64_t reqs);

// The arguments of latent_attend_rows and latent_attend_paged.
struct AttendArgs {
    bool paged;  // which of the two (ids may be null in the rows form: k == 0)
    const uint16_t *q, *cache;
    uint16_t* out;
    float* lse;                  // or nullptr
    int64_t rows, ld_q, ld_head, cache_rows, ld_cache;
    int32_t heads, d_latent;
    float scale;
    const int32_t *ids, *counts;                  // rows form
    int64_t ld_ids;
    int32_t k;
    const int32_t *query_starts, *ctx_lens;       // paged form
    int64_t reqs, max_len;
    const uint64_t* tree;
    Pages pages;
};

// How a call is cut into workgroups.
struct AttendPlan {
    int splits;       // pieces of a row's keys (at most, in the paged form), joined by a second kernel when > 1
    int groups;       // 32-row groups of query rows a workgroup
    int target;       // workgroups that the pieces are to fill
    size_t ws_bytes;  // of the pieces' results
};
AttendPlan plan_attend_rows(int64_t rows, int32_t heads, int32_t d_latent, int32_t k, bool allow_split);
AttendPlan plan_attend_paged(int64_t tokens, int64_t reqs, int32_t heads, int32_t d_latent,
                             int64_t max_len, bool allow_split);
int launch_latent_attend(const AttendArgs& a, const AttendPlan& plan, void* workspace, hipStream_t stream);

// row_limit (device, or nullptr): rows at or past *row_limit are not written.  pieces: the parts are those of
// one call's rows, where the lse of a part that saw keys, all with scores of -inf, is the lowest finite number.
// unit: what the parts' lse are in units of.
int launch_merge_attend(const void* parts, int dtype, const float* part_lse, int32_t world, int64_t rows,
                        int32_t heads, int32_t dim, void* out, int out_dtype, float* lse,
                        const int32_t* row_limit, bool pieces, float unit, hipStream_t stream);

// ------------------------------------------------------------ a beam-search step

constexpr int kMaxBeams = 64;
constexpr int kMaxBeamK = 64;
constexpr int64_t kMaxBeamRows = (1 << 24) - 1;  // groups * beams: workgroups of 256 threads in a launch

struct BeamArgs {
    const void* logits;
    const float* scores;
    float *out_scores, *ended;   // ended: or nullptr
    int32_t *parents, *tokens;
    int64_t groups, vocab, ld;   // ld in elements
    int32_t beams, k, eos;       // eos: -1 for none
    int dtype;
};

// How a call is cut: `pieces` of a row, a workgroup each, of `piece_groups` groups of 4 KB.
struct BeamPlan {
    int64_t piece_groups;
    int pieces;
    size_t ws_bytes;
    int each;  // waves of a row, where a workgroup does a whole group; 0: two launches
};
BeamPlan plan_beam_select(int dtype, int64_t groups, int32_t beams, int64_t vocab, int32_t k);
int launch_beam_select(const BeamArgs& a, const BeamPlan& plan, void* workspace, hipStream_t stream);

// The block calls hold two bits a block of the pool, and fork_blocks two words a row, in LDS.
constexpr int32_t kMaxPool = 1 << 19;
constexpr int64_t kMaxForkRows = 4096;

struct ForkArgs {
    const int32_t *table, *ctx_lens, *parents;
    const uint8_t* held;  // or nullptr
    int32_t *out_table, *out_ctx, *copies, *free_blocks, *counts;
    int64_t rows_in, ld_table, rows_out, ld_out, n_free;
    int32_t cols, block_size, pool;
};
size_t fork_blocks_bytes(int64_t rows_in, int32_t cols, int32_t pool);  // of a workspace; 0: takes none
int launch_fork_blocks(const ForkArgs& a, void* workspace, hipStream_t stream);

struct CompactArgs {
    const int32_t *table, *ctx_lens;
    const uint8_t* held;  // or nullptr
    int32_t *out_table, *moves, *free_blocks, *counts;
    int64_t rows, ld_table, ld_out, n_free, max_moves;
    int32_t cols, block_size, pool;
};
size_t compact_blocks_bytes(int64_t rows, int32_t cols, int32_t pool);
int launch_compact_blocks(const CompactArgs& a, void* workspace, hipStream_t stream);

constexpr int kMaxCopyCaches = 64;  // they travel as kernel arguments
struct CopyCache {
    char* data;
    int64_t rows, ld;          // ld in bytes
    int64_t words, row_words;  // of `word` bytes: of a block, and of a row (as many as a block's where rows follow each other)
    int64_t slice0;            // set by the launch
    int32_t word;
    int32_t lanes_log2;        // threads of a pair, set by the launch
};
template <int CACHES>
struct CopyArgs {
    const int32_t* pairs;
    int64_t n_pairs, stride_rows, slices;
    int32_t n_caches, block_size;
    CopyCache cache[CACHES];
};
int launch_copy_blocks(CopyArgs<kMaxCopyCaches>& a, hipStream_t stream);

struct KvArgs {
    const uint16_t* q;
    const void *k, *v;
    const float *k_scales, *v_scales;  // a kv head, or nullptr
    uint16_t* out;
    float* lse;  // or nullptr
    const int32_t *req_id, *row_ends;
    int64_t rows, ld_q, ld_qhead, cache_rows, ld_cache, ld_head, window, max_len;  // window: 0 for none
    int32_t heads, kv_heads, dim;
    int dtype;
    float scale;
    Pages pages;
};

constexpr int kKvLeastKeys = 64;  // of a piece
struct KvPlan {
    int target;       // pieces that the rows' keys are to be cut into, joined by a second kernel; 0: a row is one
    int rounds;       // as many times that, where they are long
    size_t ws_bytes;
};
bool kv_attend_fits(int64_t rows, int32_t heads, int32_t kv_heads);  // into a launch
KvPlan plan_kv_attend(int64_t rows, int32_t heads, int32_t kv_heads, int32_t dim, int dtype, int64_t max_len,
                      bool allow_split);
int launch_kv_attend(const KvArgs& a, const KvPlan& plan, void* workspace, hipStream_t stream);

}  // namespace rts
