// Block tables and slot maps of a batch from its requests' lengths, for gfx950.
//
// With B tokens a block, request i holds have_i = ceil(ctx_i / B) blocks and
// needs need_i = ceil((ctx_i + new_i) / B); it takes the free blocks
// [off_i, off_i + need_i - have_i), off the exclusive sum over the requests.
// Block b >= have_i starts at position b * B >= ctx_i, so the token at that
// position is new: its thread writes the table entry, and every token reads
// fresh ids from the free list instead of the table.  No workgroup reads what
// another one writes, so one launch does all of it.
//
// The work is a few bytes a token: what counts is latency.  Each workgroup
// forms both sums over all requests by itself in LDS (two block scans over at
// most 8192 entries), which costs less than a second launch would: 4 us for 64
// requests and tokens, 7 us for 509 requests and 67000 tokens.
#include "rts_device.hpp"
#include "rts_internal.h"
#include "../../include/row_top_select.h"

namespace rts {

constexpr int kSlotBlock = 256;
constexpr int kSlotWaves = kSlotBlock / kWave;

// Turns v[0, n) in LDS into its exclusive sums, capped at `cap`, and returns
// the whole sum (not capped).  Sums are held in 64 bits.
template <typename Load>
__device__ __forceinline__ int64_t block_sums(int n, Load&& load, int64_t cap, int32_t* v, int64_t* wave_sum) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int per = (n + kSlotBlock - 1) / kSlotBlock;
    const int lo = tid * per < n ? tid * per : n, hi = lo + per < n ? lo + per : n;
    int64_t own = 0;
    for (int i = lo; i < hi; ++i) own += load(i);
    int64_t inc = own;
    for (int d = 1; d < kWave; d <<= 1) {
        const int64_t up = __shfl_up(inc, d);
        if (lane >= d) inc += up;
    }
    if (lane == kWave - 1) wave_sum[wave] = inc;
    __syncthreads();
    int64_t before = inc - own, total = 0;
    for (int w = 0; w < kSlotWaves; ++w) {
        if (w < wave) before += wave_sum[w];
        total += wave_sum[w];
    }
    for (int i = lo; i < hi; ++i) {
        const int64_t x = load(i);  // before v[i] is written: load may read it
        v[i] = (int32_t)(before < cap ? before : cap);
        before += x;
    }
    __syncthreads();
    return total;
}

__global__ __launch_bounds__(kSlotBlock) void assign_slots_kernel(
    const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ new_lens, int reqs, int64_t tokens,
    int32_t block_size, int64_t stride_rows, const int32_t* __restrict__ free_blocks, int64_t free_count,
    int32_t* __restrict__ table, int32_t table_cols, int64_t ld_table, int32_t* __restrict__ query_starts,
    int32_t* __restrict__ req_id, int32_t* __restrict__ row_ends, int32_t* __restrict__ slots,
    int32_t* __restrict__ used) {
    extern __shared__ int32_t lds[];
    int32_t* starts = lds;              // [reqs + 1] first token of each request
    int32_t* off = lds + reqs + 1;      // [reqs] first free block of each request
    __shared__ int64_t wave_sum[2][kSlotWaves];
    const int tid = threadIdx.x;
    const int64_t bs = block_size;
    auto ctx_of = [&](int i) { const int32_t c = ctx_lens[i]; return (int64_t)(c > 0 ? c : 0); };

    const int64_t sum = block_sums(
        reqs, [&](int i) { const int32_t n = new_lens[i]; return (int64_t)(n > 0 ? n : 0); }, tokens,
        starts, wave_sum[0]);
    const int32_t total = (int32_t)(sum < tokens ? sum : tokens);
    if (tid == 0) starts[reqs] = total;
    __syncthreads();
    const int64_t taken = block_sums(
        reqs,
        [&](int i) {
            const int64_t c = ctx_of(i), n = starts[i + 1] - starts[i];
            return (c + n + bs - 1) / bs - (c + bs - 1) / bs;
        },
        free_count, off, wave_sum[1]);

    const int64_t at = (int64_t)blockIdx.x * kSlotBlock + tid;
    const int64_t step = (int64_t)gridDim.x * kSlotBlock;
    for (int64_t i = at; i <= reqs; i += step) query_starts[i] = starts[i];
    if (at == 0) used[0] = (int32_t)(taken < 0x7FFFFFFFll ? taken : 0x7FFFFFFFll);
    for (int64_t t = at; t < tokens; t += step) {
        if (t >= total) {
            req_id[t] = -1;
            row_ends[t] = 0;
            slots[t] = -1;
            continue;
        }
        int lo = 0, hi = reqs;  // the last request that starts at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (starts[mid] <= t) lo = mid; else hi = mid;
        }
        const int64_t ctx = ctx_of(lo), pos = ctx + t - starts[lo];
        const int64_t b = pos / bs, in = pos - b * bs, have = (ctx + bs - 1) / bs;
        int32_t id = -1;
        if (b >= have) {
            const int64_t f = off[lo] + (b - have);
            if (f < free_count) id = free_blocks[f];
            if (in == 0 && b < table_cols) table[lo * ld_table + b] = id;
        }
        if (b >= table_cols) id = -1;
        else if (b < have) id = table[lo * ld_table + b];
        req_id[t] = lo;
        row_ends[t] = (int32_t)(pos + 1 < 0x7FFFFFFFll ? pos + 1 : 0x7FFFFFFFll);
        slots[t] = id < 0 ? -1 : (int32_t)((uint32_t)id * (uint32_t)stride_rows + (uint32_t)in);  // the low 32 bits
    }
}

int launch_assign_slots(const int32_t* ctx_lens, const int32_t* new_lens, int64_t reqs, int64_t tokens,
                        int32_t block_size, int64_t stride_rows, const int32_t* free_blocks,
                        int64_t free_count, int32_t* block_table, int32_t table_cols, int64_t ld_table,
                        int32_t* query_starts, int32_t* req_id, int32_t* row_ends, int32_t* slots,
                        int32_t* used, hipStream_t s) {
    const int64_t want = ((tokens > reqs ? tokens : reqs + 1) + kSlotBlock - 1) / kSlotBlock;
    const int64_t blocks = want < 1024 ? want : 1024;
    const size_t lds = (size_t)(2 * reqs + 1) * sizeof(int32_t);
    hipLaunchKernelGGL(assign_slots_kernel, dim3((unsigned)blocks), dim3(kSlotBlock), lds, s, ctx_lens,
                       new_lens, (int)reqs, tokens, block_size, stride_rows, free_blocks, free_count,
                       block_table, table_cols, ld_table, query_starts, req_id, row_ends, slots, used);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

}  // namespace rts
