// The C ABI of row_top_select: argument validation on the host (nothing is
// launched on a bad call, in the spirit of the host checks of _check_exact on
// the kernels page of vllm.models.kimi_k3.nvidia.ops.dcp_topk_merge), then the
// launchers next to the kernels.  No allocation, no synchronisation.
#include "../../include/row_top_select.h"

#include <stdint.h>

#include <cmath>

#include "rts_internal.h"

namespace {

constexpr int32_t kMaxK = 2048;
constexpr int64_t kMaxGrid = 0x7FFFFFFFll;
constexpr int64_t kMaxCandidates = 32768;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" {

const char* rts_status_string(int status) {
    switch (status) {
        case RTS_OK: return "RTS_OK";
        case RTS_EINVAL: return "RTS_EINVAL: invalid argument";
        case RTS_EUNSUPPORTED: return "RTS_EUNSUPPORTED: request outside this build's limits";
        case RTS_EWORKSPACE: return "RTS_EWORKSPACE: workspace smaller than required";
        case RTS_EHIP: return "RTS_EHIP: HIP launch failed";
        default: return "unknown rts_status";
    }
}

size_t topk_rows_workspace_size(int dtype, int64_t rows, int64_t cols, int32_t k) {
    if ((dtype != RTS_F32 && dtype != RTS_BF16) || rows < 0 || cols < 0 || k < 1 || k > kMaxK)
        return 0;
    return rts::plan_topk_rows(dtype, rows, cols, k, true).ws_bytes;
}

int topk_rows(const void* logits, int dtype, int64_t rows, int64_t cols, int64_t ld_logits,
              const int32_t* row_ends, int32_t k, int32_t* out_idx, int64_t ld_out, void* workspace,
              size_t workspace_bytes, hipStream_t stream) {
    if (dtype != RTS_F32 && dtype != RTS_BF16) return RTS_EINVAL;
    if (rows < 0 || cols < 0 || ld_logits < cols || ld_logits < 0 || k < 1 || ld_out < k)
        return RTS_EINVAL;
    if (k > kMaxK || cols > 0x7FFFFFFFll) return RTS_EUNSUPPORTED;
    if (rows == 0) return RTS_OK;
    if (!out_idx || (cols > 0 && !logits)) return RTS_EINVAL;
    const size_t esz = dtype == RTS_F32 ? 4 : 2;
    if (!aligned(logits, esz) || !aligned(out_idx, 4) || (row_ends && !aligned(row_ends, 4)))
        return RTS_EINVAL;
    if (workspace_bytes > 0 && !workspace) return RTS_EINVAL;
    const bool have_ws = workspace != nullptr;
    rts::TopkPlan plan = rts::plan_topk_rows(dtype, rows, cols, k, have_ws);
    if (have_ws && workspace_bytes < plan.ws_bytes) return RTS_EWORKSPACE;
    if (have_ws && !aligned(workspace, 8)) return RTS_EINVAL;
    if (rows * plan.groups > kMaxGrid) return RTS_EUNSUPPORTED;
    return rts::launch_topk_rows(logits, dtype, rows, cols, ld_logits, row_ends, k, out_idx, ld_out,
                                 plan, workspace, stream);
}

int topk_rows_noalloc(const void* logits, int dtype, int64_t rows, int64_t cols, int64_t ld_logits,
                      const int32_t* row_ends, int32_t k, int32_t* out_idx, int64_t ld_out,
                      hipStream_t stream) {
    if (dtype != RTS_F32 && dtype != RTS_BF16) return RTS_EINVAL;
    if (rows < 0 || cols < 0 || ld_logits < cols || ld_logits < 0 || k < 1 || ld_out < k)
        return RTS_EINVAL;
    if (k > kMaxK || cols > 0x7FFFFFFFll) return RTS_EUNSUPPORTED;
    if (rows == 0) return RTS_OK;
    if (!out_idx || (cols > 0 && !logits)) return RTS_EINVAL;
    const size_t esz = dtype == RTS_F32 ? 4 : 2;
    if (!aligned(logits, esz) || !aligned(out_idx, 4) || (row_ends && !aligned(row_ends, 4)))
        return RTS_EINVAL;
    rts::TopkPlan plan = rts::plan_topk_rows(dtype, rows, cols, k, true);
    void* scratch = nullptr;
    if (plan.groups > 1) {
        size_t bytes = 0;
        const int rc = rts::scratch_of_current_device(&scratch, &bytes);
        if (rc != RTS_OK) return rc;
        if (plan.ws_bytes > bytes) return RTS_EWORKSPACE;
    }
    if (rows * plan.groups > kMaxGrid) return RTS_EUNSUPPORTED;
    return rts::launch_topk_rows(logits, dtype, rows, cols, ld_logits, row_ends, k, out_idx, ld_out,
                                 plan, scratch, stream);
}

int pack_candidates(const uint16_t* logits_bf16, int64_t rows, int64_t cols, int64_t ld_logits,
                    const int32_t* local_idx, int32_t n, int64_t ld_idx, const int32_t* row_ends,
                    int32_t* packed, hipStream_t stream) {
    if (rows < 0 || cols < 0 || ld_logits < cols || n < 32 || n % 32 != 0 || ld_idx < n)
        return RTS_EINVAL;
    if (rows == 0) return RTS_OK;
    if (!logits_bf16 || !local_idx || !packed) return RTS_EINVAL;
    if (!aligned(logits_bf16, 2) || !aligned(local_idx, 4) || !aligned(packed, 4) ||
        (row_ends && !aligned(row_ends, 4)))
        return RTS_EINVAL;
    if ((rows * (int64_t)n + 255) / 256 > kMaxGrid) return RTS_EUNSUPPORTED;
    return rts::launch_pack_candidates(logits_bf16, rows, cols, ld_logits, local_idx, n, ld_idx,
                                       row_ends, packed, stream);
}

namespace {
int merge_packed_checked(const int32_t* gathered, bool row_major, int32_t world, int64_t rows,
                         int32_t n, int32_t k, int32_t* out_ids, int32_t* sat_word,
                         hipStream_t stream) {
    if (world < 1 || world > 16 || rows < 0 || n < 32 || n % 32 != 0 || k < 1) return RTS_EINVAL;
    if (k > kMaxK || (int64_t)world * n > kMaxCandidates || rows > kMaxGrid) return RTS_EUNSUPPORTED;
    if (rows == 0) return RTS_OK;
    if (!gathered || !out_ids) return RTS_EINVAL;
    if (!aligned(gathered, 4) || !aligned(out_ids, 4) || (sat_word && !aligned(sat_word, 4)))
        return RTS_EINVAL;
    return rts::launch_merge_packed(gathered, row_major, world, rows, n, k, out_ids, sat_word, nullptr,
                                    stream);
}

int merge_pairs_checked(const int32_t* gathered_pairs, bool row_major, int32_t world, int64_t rows,
                        int32_t kc, int32_t k, int32_t* out_ids, hipStream_t stream) {
    if (world < 1 || rows < 0 || kc < 1 || k < 1) return RTS_EINVAL;
    if (k > kMaxK || (int64_t)world * kc > kMaxCandidates || rows > kMaxGrid) return RTS_EUNSUPPORTED;
    if (rows == 0) return RTS_OK;
    if (!gathered_pairs || !out_ids) return RTS_EINVAL;
    if (!aligned(gathered_pairs, 8) || !aligned(out_ids, 4)) return RTS_EINVAL;
    return rts::launch_merge_pairs(gathered_pairs, row_major, world, rows, kc, k, out_ids, stream);
}
}  // namespace

int merge_select_rank_major(const int32_t* gathered, int32_t world, int64_t rows, int32_t n,
                            int32_t k, int32_t* out_ids, int32_t* sat_word, hipStream_t stream) {
    return merge_packed_checked(gathered, false, world, rows, n, k, out_ids, sat_word, stream);
}

int merge_select_row_major(const int32_t* gathered, int32_t world, int64_t rows, int32_t n, int32_t k,
                           int32_t* out_ids, int32_t* sat_word, hipStream_t stream) {
    return merge_packed_checked(gathered, true, world, rows, n, k, out_ids, sat_word, stream);
}

int rescue_push(const int32_t* local_packed, int32_t rank, int32_t world, int64_t rows, int32_t n,
                int32_t k, const int32_t* sat_word, int32_t* recv, hipStream_t stream) {
    if (world < 1 || world > 16 || rank < 0 || rank >= world || rows < 0 || n < 32 || n % 32 != 0 ||
        k < 32 || k % 32 != 0)
        return RTS_EINVAL;
    if (k > kMaxK || (rows + 3) / 4 > kMaxGrid) return RTS_EUNSUPPORTED;
    if (rows == 0 || (k - 1) / n == 0) return RTS_OK;
    if (!local_packed || !sat_word || !recv) return RTS_EINVAL;
    if (!aligned(local_packed, 4) || !aligned(sat_word, 4) || !aligned(recv, 4)) return RTS_EINVAL;
    return rts::launch_rescue_push(local_packed, rank, world, rows, n, k, sat_word, recv, stream);
}

int merge_rescue_rank_major(const int32_t* gathered, const int32_t* recv, int32_t world, int64_t rows,
                            int32_t n, int32_t k, const int32_t* sat_word, int32_t* out_ids,
                            hipStream_t stream) {
    if (world < 1 || world > 16 || rows < 0 || n < 32 || n % 32 != 0 || k < 32 || k % 32 != 0)
        return RTS_EINVAL;
    if (k > kMaxK || rts::rescue_candidates(world, n, k) > kMaxCandidates || rows > kMaxGrid)
        return RTS_EUNSUPPORTED;
    if (rows == 0 || (k - 1) / n == 0) return RTS_OK;
    if (!gathered || !recv || !sat_word || !out_ids) return RTS_EINVAL;
    if (!aligned(gathered, 4) || !aligned(recv, 4) || !aligned(sat_word, 4) || !aligned(out_ids, 4))
        return RTS_EINVAL;
    return rts::launch_merge_rescue(gathered, recv, world, rows, n, k, sat_word, out_ids, nullptr, stream);
}

int emit_rows(const int32_t* ids, int64_t rows, int32_t k, int32_t world, int32_t dcp_rank,
              const int32_t* req_id, const int32_t* block_table, int64_t table_rows, int32_t table_cols,
              int64_t ld_table, int32_t block_size, int64_t stride_rows, int32_t* rows_out,
              int32_t out_cols, int32_t* valid_out, hipStream_t stream) {
    if (rows < 0 || k < 1 || world < 1 || dcp_rank < 0 || dcp_rank >= world || table_rows < 0 ||
        table_cols < 0 || ld_table < table_cols || block_size < 1 || out_cols < k)
        return RTS_EINVAL;
    if (k > kMaxK || (rows + 3) / 4 > kMaxGrid) return RTS_EUNSUPPORTED;
    if (rows == 0) return RTS_OK;
    if (!ids || !req_id || !rows_out || !valid_out || (table_rows > 0 && table_cols > 0 && !block_table))
        return RTS_EINVAL;
    if (!aligned(ids, 4) || !aligned(req_id, 4) || !aligned(rows_out, 4) || !aligned(valid_out, 4) ||
        (block_table && !aligned(block_table, 4)))
        return RTS_EINVAL;
    return rts::launch_emit_rows(ids, rows, k, world, dcp_rank, req_id, block_table, table_rows,
                                 table_cols, ld_table, block_size, stride_rows, rows_out, out_cols,
                                 valid_out, stream);
}

namespace {
// Validates an rts_kv_rows against k and world and converts it.
int kv_rows_args(const rts_kv_rows* kv, int32_t k, int32_t world, rts::RowsArgs& ra) {
    if (!kv || kv->dcp_rank < 0 || kv->dcp_rank >= world || kv->table_rows < 0 || kv->table_cols < 0 ||
        kv->ld_table < kv->table_cols || kv->block_size < 1 || kv->out_cols < k)
        return RTS_EINVAL;
    if (!kv->req_id || !kv->rows_out || !kv->valid_out ||
        (kv->table_rows > 0 && kv->table_cols > 0 && !kv->block_table))
        return RTS_EINVAL;
    if (!aligned(kv->req_id, 4) || !aligned(kv->rows_out, 4) || !aligned(kv->valid_out, 4) ||
        (kv->block_table && !aligned(kv->block_table, 4)))
        return RTS_EINVAL;
    ra = rts::RowsArgs{kv->req_id, kv->block_table, kv->rows_out, kv->valid_out, kv->table_rows,
                       kv->ld_table, kv->stride_rows, kv->dcp_rank, kv->table_cols, kv->block_size,
                       kv->out_cols};
    return RTS_OK;
}
}  // namespace

int merge_select_rank_major_rows(const int32_t* gathered, int32_t world, int64_t rows, int32_t n,
                                 int32_t k, const rts_kv_rows* kv, int32_t* out_ids, int32_t* sat_word,
                                 hipStream_t stream) {
    if (world < 1 || world > 16 || rows < 0 || n < 32 || n % 32 != 0 || k < 1) return RTS_EINVAL;
    if (k > kMaxK || (int64_t)world * n > kMaxCandidates || rows > kMaxGrid) return RTS_EUNSUPPORTED;
    rts::RowsArgs ra;
    const int rc = kv_rows_args(kv, k, world, ra);
    if (rc != RTS_OK) return rc;
    if (rows == 0) return RTS_OK;
    if (!gathered || !aligned(gathered, 4) || (out_ids && !aligned(out_ids, 4)) ||
        (sat_word && !aligned(sat_word, 4)))
        return RTS_EINVAL;
    return rts::launch_merge_packed(gathered, false, world, rows, n, k, out_ids, sat_word, &ra, stream);
}

int merge_rescue_rank_major_rows(const int32_t* gathered, const int32_t* recv, int32_t world,
                                 int64_t rows, int32_t n, int32_t k, const int32_t* sat_word,
                                 const rts_kv_rows* kv, int32_t* out_ids, hipStream_t stream) {
    if (world < 1 || world > 16 || rows < 0 || n < 32 || n % 32 != 0 || k < 32 || k % 32 != 0)
        return RTS_EINVAL;
    if (k > kMaxK || rts::rescue_candidates(world, n, k) > kMaxCandidates || rows > kMaxGrid)
        return RTS_EUNSUPPORTED;
    rts::RowsArgs ra;
    const int rc = kv_rows_args(kv, k, world, ra);
    if (rc != RTS_OK) return rc;
    if (rows == 0 || (k - 1) / n == 0) return RTS_OK;
    if (!gathered || !recv || !sat_word) return RTS_EINVAL;
    if (!aligned(gathered, 4) || !aligned(recv, 4) || !aligned(sat_word, 4) ||
        (out_ids && !aligned(out_ids, 4)))
        return RTS_EINVAL;
    return rts::launch_merge_rescue(gathered, recv, world, rows, n, k, sat_word, out_ids, &ra, stream);
}

int pack_pairs(const float* logits, int64_t rows, int64_t cols, int64_t ld_logits,
               const int32_t* local_idx, int32_t kc, int64_t ld_idx, const int32_t* row_ends,
               int32_t rank, int32_t world, int32_t* pairs, hipStream_t stream) {
    if (rows < 0 || cols < 0 || ld_logits < cols || kc < 1 || ld_idx < kc || world < 1 ||
        rank < 0 || rank >= world)
        return RTS_EINVAL;
    if (cols * (int64_t)world > 0x7FFFFFFFll) return RTS_EUNSUPPORTED;
    if (rows == 0) return RTS_OK;
    if (!logits || !local_idx || !pairs) return RTS_EINVAL;
    if (!aligned(logits, 4) || !aligned(local_idx, 4) || !aligned(pairs, 8) ||
        (row_ends && !aligned(row_ends, 4)))
        return RTS_EINVAL;
    if ((rows * (int64_t)kc + 255) / 256 > kMaxGrid) return RTS_EUNSUPPORTED;
    return rts::launch_pack_pairs(logits, rows, cols, ld_logits, local_idx, kc, ld_idx, row_ends,
                                  rank, world, pairs, stream);
}

int merge_select_pairs_rank_major(const int32_t* gathered_pairs, int32_t world, int64_t rows,
                                  int32_t kc, int32_t k, int32_t* out_ids, hipStream_t stream) {
    return merge_pairs_checked(gathered_pairs, false, world, rows, kc, k, out_ids, stream);
}

int merge_select_pairs_row_major(const int32_t* gathered_pairs, int32_t world, int64_t rows,
                                 int32_t kc, int32_t k, int32_t* out_ids, hipStream_t stream) {
    return merge_pairs_checked(gathered_pairs, true, world, rows, kc, k, out_ids, stream);
}

int assign_slots(const int32_t* ctx_lens, const int32_t* new_lens, int64_t reqs, int64_t tokens,
                 int32_t block_size, int64_t stride_rows, const int32_t* free_blocks,
                 int64_t free_count, int32_t* block_table, int32_t table_cols, int64_t ld_table,
                 int32_t* query_starts, int32_t* req_id, int32_t* row_ends, int32_t* slots,
                 int32_t* used, hipStream_t stream) {
    if (reqs < 0 || tokens < 0 || block_size < 1 || stride_rows < 0 || free_count < 0 ||
        table_cols < 0 || ld_table < table_cols)
        return RTS_EINVAL;
    if (reqs > rts::kMaxReqs || tokens > 0x7FFFFFFFll || free_count > 0x7FFFFFFFll)
        return RTS_EUNSUPPORTED;
    if (!query_starts || !used || (reqs > 0 && (!ctx_lens || !new_lens)) ||
        (tokens > 0 && (!req_id || !row_ends || !slots)) || (free_count > 0 && !free_blocks) ||
        (reqs > 0 && table_cols > 0 && !block_table))
        return RTS_EINVAL;
    if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(free_blocks, 4) ||
        !aligned(block_table, 4) || !aligned(query_starts, 4) || !aligned(req_id, 4) ||
        !aligned(row_ends, 4) || !aligned(slots, 4) || !aligned(used, 4))
        return RTS_EINVAL;
    return rts::launch_assign_slots(ctx_lens, new_lens, reqs, tokens, block_size, stride_rows, free_blocks,
                                    free_count, block_table, table_cols, ld_table, query_starts, req_id,
                                    row_ends, slots, used, stream);
}

namespace {
// What indexer_logits and indexer_logits_paged check alike.
int logits_args(const rts::LogitsArgs& a) {
    if (a.dtype != RTS_BF16 && a.dtype != RTS_E4M3) return RTS_EINVAL;
    if (a.logits_dtype != RTS_F32 && a.logits_dtype != RTS_BF16) return RTS_EINVAL;
    if (a.rows < 0 || a.cols < 0 || a.heads < 1 || a.dim < 1 || a.ld_weights < a.heads ||
        a.ld_logits < a.cols || a.ld_keys < a.dim || a.ld_q < (int64_t)a.heads * a.dim)
        return RTS_EINVAL;
    if (a.heads > 128 || (a.dim != 64 && a.dim != 128) || a.cols > 0x7FFFFFFFll ||
        a.rows > 0x7FFFFFFFll || a.ld_keys > (1 << 30))
        return RTS_EUNSUPPORTED;
    if (a.rows == 0 || a.cols == 0) return RTS_OK;
    const int64_t esz = a.dtype == RTS_BF16 ? 2 : 1;
    if (!a.q || !a.weights || !a.logits) return RTS_EINVAL;
    if (!aligned(a.q, 16) || !aligned(a.keys, 16) || a.ld_q * esz % 16 != 0 || a.ld_keys * esz % 16 != 0 ||
        !aligned(a.weights, 4) || !aligned(a.key_scales, 4) || !aligned(a.row_ends, 4) ||
        !aligned(a.logits, a.logits_dtype == RTS_F32 ? 4 : 2))
        return RTS_EINVAL;
    return RTS_OK;
}

int pages_args(const int32_t* block_table, int64_t table_rows, int32_t table_cols, int64_t ld_table,
               int32_t block_size, int64_t stride_rows, int64_t cache_rows) {
    if (table_rows < 0 || table_cols < 0 || ld_table < table_cols || block_size < 1 || stride_rows < 0 ||
        cache_rows < 0 || !aligned(block_table, 4) || (table_rows > 0 && table_cols > 0 && !block_table))
        return RTS_EINVAL;
    return RTS_OK;
}
}  // namespace

int indexer_logits(const void* q, int dtype, int64_t rows, int32_t heads, int32_t dim, int64_t ld_q,
                   const void* keys, int64_t cols, int64_t ld_keys, const float* weights,
                   int64_t ld_weights, const float* key_scales, const int32_t* row_ends, void* logits,
                   int logits_dtype, int64_t ld_logits, hipStream_t stream) {
    rts::LogitsArgs a{};
    a.q = q, a.keys = keys, a.weights = weights, a.key_scales = key_scales, a.row_ends = row_ends;
    a.logits = logits, a.rows = rows, a.cols = cols, a.ld_q = ld_q, a.ld_keys = ld_keys;
    a.ld_weights = ld_weights, a.ld_logits = ld_logits, a.heads = heads, a.dim = dim;
    a.dtype = dtype, a.logits_dtype = logits_dtype;
    const int rc = logits_args(a);
    if (rc != RTS_OK) return rc;
    if (rows == 0 || cols == 0) return RTS_OK;
    if (!keys) return RTS_EINVAL;
    return rts::launch_indexer_logits(a, stream);
}

int indexer_logits_paged(const void* q, int dtype, int64_t rows, int32_t heads, int32_t dim,
                         int64_t ld_q, const void* key_cache, int64_t cache_rows, int64_t ld_keys,
                         const float* weights, int64_t ld_weights, const float* key_scales,
                         const int32_t* req_id, const int32_t* row_ends, const int32_t* block_table,
                         int64_t table_rows, int32_t table_cols, int64_t ld_table, int32_t block_size,
                         int64_t stride_rows, int64_t cols, void* logits, int logits_dtype,
                         int64_t ld_logits, hipStream_t stream) {
    rts::LogitsArgs a{};
    a.q = q, a.keys = key_cache, a.weights = weights, a.key_scales = key_scales, a.row_ends = row_ends;
    a.req_id = req_id, a.logits = logits, a.rows = rows, a.cols = cols, a.ld_q = ld_q;
    a.ld_keys = ld_keys, a.ld_weights = ld_weights, a.ld_logits = ld_logits, a.heads = heads;
    a.dim = dim, a.dtype = dtype, a.logits_dtype = logits_dtype;
    int rc = logits_args(a);
    if (rc != RTS_OK) return rc;
    rc = pages_args(block_table, table_rows, table_cols, ld_table, block_size, stride_rows, cache_rows);
    if (rc != RTS_OK) return rc;
    if (cache_rows > 0x7FFFFFFFll) return RTS_EUNSUPPORTED;
    if (rows == 0 || cols == 0) return RTS_OK;
    if (!req_id || !row_ends || !aligned(req_id, 4) || (cache_rows > 0 && !key_cache)) return RTS_EINVAL;
    a.pages = rts::make_pages(block_table, table_rows, table_cols, ld_table, block_size, stride_rows,
                              cache_rows);
    return rts::launch_indexer_logits(a, stream);
}

int indexer_logits_plan(int dtype, int64_t rows, int32_t heads, int32_t dim, int64_t cols, int64_t table_rows,
                        int64_t* plan) {
    if ((dtype != RTS_BF16 && dtype != RTS_E4M3) || rows < 1 || cols < 1 || heads < 1 || table_rows < -1 || !plan)
        return RTS_EINVAL;
    if (heads > 128 || (dim != 64 && dim != 128) || cols > 0x7FFFFFFFll || rows > 0x7FFFFFFFll)
        return RTS_EUNSUPPORTED;
    const rts::LogitsPlan p = rts::plan_indexer_logits(dtype, rows, cols, heads, dim, table_rows);
    plan[0] = p.tokens, plan[1] = p.steps, plan[2] = p.step, plan[3] = p.stages;
    return RTS_OK;
}

namespace {
// What latent_attend_rows and latent_attend_paged check alike.
int attend_args(const rts::AttendArgs& a, int32_t d_rope) {
    if (a.rows < 0 || a.heads < 1 || a.d_latent < 1 || d_rope < 0 || a.cache_rows < 0) return RTS_EINVAL;
    const int64_t d = (int64_t)a.d_latent + d_rope;
    if (a.ld_cache < d || a.ld_head < d || a.ld_q < 0 || !(std::fabs(a.scale) <= 0x1p127f)) return RTS_EINVAL;
    if ((a.d_latent != 256 && a.d_latent != 512) || d_rope != 64 || a.heads > 1024 ||
        a.rows > 0x7FFFFFFFll / a.heads || a.cache_rows > 0x7FFFFFFFll)
        return RTS_EUNSUPPORTED;
    if (a.rows == 0) return RTS_OK;
    if (!a.q || !a.out || (a.cache_rows > 0 && !a.cache)) return RTS_EINVAL;
    if (!aligned(a.q, 16) || !aligned(a.cache, 16) || !aligned(a.out, 16) || a.ld_q % 8 != 0 ||
        a.ld_head % 8 != 0 || a.ld_cache % 8 != 0 || !aligned(a.lse, 4))
        return RTS_EINVAL;
    return RTS_OK;
}

int attend_planned(const rts::AttendArgs& a, const rts::AttendPlan& plan, void* workspace,
                   size_t workspace_bytes, hipStream_t stream) {
    if (workspace && workspace_bytes < plan.ws_bytes) return RTS_EWORKSPACE;
    if (workspace && !aligned(workspace, 16)) return RTS_EINVAL;
    return rts::launch_latent_attend(a, plan, workspace, stream);
}
}  // namespace

size_t latent_attend_rows_workspace_size(int64_t rows, int32_t heads, int32_t d_latent, int32_t k) {
    if (rows < 1 || heads < 1 || heads > 1024 || rows > 0x7FFFFFFFll / heads || k < 0 ||
        (d_latent != 256 && d_latent != 512))
        return 0;
    return rts::plan_attend_rows(rows, heads, d_latent, k, true).ws_bytes;
}

int latent_attend_rows(const void* q, int64_t rows, int32_t heads, int32_t d_latent, int32_t d_rope,
                       int64_t ld_q, int64_t ld_head, const void* cache, int64_t cache_rows,
                       int64_t ld_cache, const int32_t* ids, int32_t k, int64_t ld_ids,
                       const int32_t* counts, float scale, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
    rts::AttendArgs a{};
    a.paged = false;
    a.q = static_cast<const uint16_t*>(q), a.cache = static_cast<const uint16_t*>(cache);
    a.out = static_cast<uint16_t*>(out), a.lse = lse, a.rows = rows, a.ld_q = ld_q, a.ld_head = ld_head;
    a.cache_rows = cache_rows, a.ld_cache = ld_cache, a.heads = heads, a.d_latent = d_latent;
    a.scale = scale, a.ids = ids, a.counts = counts, a.ld_ids = ld_ids, a.k = k;
    if (k < 0 || ld_ids < k || (workspace_bytes > 0 && !workspace)) return RTS_EINVAL;
    const int rc = attend_args(a, d_rope);
    if (rc != RTS_OK) return rc;
    if (rows == 0) return RTS_OK;
    if ((k > 0 && !ids) || !aligned(ids, 4) || !aligned(counts, 4)) return RTS_EINVAL;
    return attend_planned(a, rts::plan_attend_rows(rows, heads, d_latent, k, workspace != nullptr),
                          workspace, workspace_bytes, stream);
}

int latent_attend_rows_plan(int64_t rows, int32_t heads, int32_t d_latent, int32_t k, int split, int32_t* plan) {
    if (rows < 1 || heads < 1 || k < 0 || !plan) return RTS_EINVAL;
    if (heads > 1024 || rows > 0x7FFFFFFFll / heads || (d_latent != 256 && d_latent != 512)) return RTS_EUNSUPPORTED;
    const rts::AttendPlan p = rts::plan_attend_rows(rows, heads, d_latent, k, split != 0);
    plan[0] = p.groups, plan[1] = p.splits;
    return RTS_OK;
}

int latent_attend_paged_plan(int64_t tokens, int64_t reqs, int32_t heads, int32_t d_latent, int64_t max_len,
                             int split, int32_t* plan) {
    if (tokens < 1 || reqs < 1 || heads < 1 || max_len < 0 || !plan) return RTS_EINVAL;
    if (heads > 1024 || tokens > 0x7FFFFFFFll / heads || (d_latent != 256 && d_latent != 512)) return RTS_EUNSUPPORTED;
    const rts::AttendPlan p = rts::plan_attend_paged(tokens, reqs, heads, d_latent, max_len, split != 0);
    plan[0] = p.groups, plan[1] = p.splits;
    return RTS_OK;
}

size_t latent_attend_paged_workspace_size(int64_t tokens, int64_t reqs, int32_t heads,
                                          int32_t d_latent, int64_t max_len) {
    if (tokens < 1 || reqs < 1 || heads < 1 || heads > 1024 || tokens > 0x7FFFFFFFll / heads ||
        max_len < 0 || (d_latent != 256 && d_latent != 512))
        return 0;
    return rts::plan_attend_paged(tokens, reqs, heads, d_latent, max_len, true).ws_bytes;
}

int latent_attend_paged(const void* q, int64_t tokens, int32_t heads, int32_t d_latent,
                        int32_t d_rope, int64_t ld_q, int64_t ld_head, const void* cache,
                        int64_t cache_rows, int64_t ld_cache, const int32_t* query_starts,
                        const int32_t* ctx_lens, int64_t reqs, const uint64_t* tree,
                        const int32_t* block_table, int32_t table_cols, int64_t ld_table,
                        int32_t block_size, int64_t stride_rows, int64_t max_len, float scale,
                        void* out, float* lse, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
    rts::AttendArgs a{};
    a.paged = true;
    a.q = static_cast<const uint16_t*>(q), a.cache = static_cast<const uint16_t*>(cache);
    a.out = static_cast<uint16_t*>(out), a.lse = lse, a.rows = tokens, a.ld_q = ld_q, a.ld_head = ld_head;
    a.cache_rows = cache_rows, a.ld_cache = ld_cache, a.heads = heads, a.d_latent = d_latent;
    a.scale = scale, a.query_starts = query_starts, a.ctx_lens = ctx_lens, a.reqs = reqs;
    a.max_len = max_len, a.tree = tree;
    if (reqs < 0 || max_len < 0 || (workspace_bytes > 0 && !workspace)) return RTS_EINVAL;
    int rc = attend_args(a, d_rope);
    if (rc != RTS_OK) return rc;
    rc = pages_args(block_table, reqs, table_cols, ld_table, block_size, stride_rows, cache_rows);
    if (rc != RTS_OK) return rc;
    if (reqs > 0x7FFFFFFFll - tokens * heads) return RTS_EUNSUPPORTED;
    if (tokens == 0 || reqs == 0) return RTS_OK;
    if (!query_starts || !ctx_lens || !aligned(query_starts, 4) || !aligned(ctx_lens, 4) ||
        !aligned(tree, 8))
        return RTS_EINVAL;
    a.pages = rts::make_pages(block_table, reqs, table_cols, ld_table, block_size, stride_rows, cache_rows);
    return attend_planned(a, rts::plan_attend_paged(tokens, reqs, heads, d_latent, max_len,
                                                    workspace != nullptr),
                          workspace, workspace_bytes, stream);
}

int merge_attend_rank_major(const void* parts, int dtype, const float* part_lse, int32_t world,
                            int64_t rows, int32_t heads, int32_t dim, void* out, int out_dtype,
                            float* lse, hipStream_t stream) {
    if ((dtype != RTS_F32 && dtype != RTS_BF16) || (out_dtype != RTS_F32 && out_dtype != RTS_BF16))
        return RTS_EINVAL;
    if (world < 1 || world > 64 || rows < 0 || heads < 1 || dim < 8 || dim % 8 != 0) return RTS_EINVAL;
    if (dim > 2048 || rows > 0x7FFFFFFFll / heads) return RTS_EUNSUPPORTED;
    if (rows == 0) return RTS_OK;
    if (!parts || !part_lse || !out) return RTS_EINVAL;
    if (!aligned(parts, 16) || !aligned(out, 16) || !aligned(part_lse, 4) || !aligned(lse, 4))
        return RTS_EINVAL;
    return rts::launch_merge_attend(parts, dtype, part_lse, world, rows, heads, dim, out, out_dtype, lse,
                                    nullptr, false, stream);
}

}  // extern "C"
