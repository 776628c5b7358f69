// Forking, freeing, compacting and copying the blocks of a paged cache, for
// gfx950.
//
// Which blocks are in use is not kept anywhere: it follows from the block
// tables and lengths, one bit a block.  Every workgroup forms these bits for
// the whole pool by itself in LDS (64 KB for 2^19 blocks), takes the ranks that
// it needs from them and writes its share of the outputs, so that no workgroup
// reads what another one writes and one launch does all of it.  (Counters kept from
// call to call would be state to lose, and atomic ones an order to depend on.)  The work is a
// few bytes a block and table entry: what counts is the chain of steps, and on large tables
// that each workgroup reads them.  Those are read by workgroups of their own first, see mark_parts.
//
// Measured, kernels: fork_blocks 256 x 257 entries, 74240 blocks: 15.7 us (marking 7, the
// ranks 3, the tables 2); 800 x 513, 462400 blocks: 8.6 + 3.3 + 12.8; compact_blocks 64 x 129:
// 10.1; 1000 x 257, 386000 blocks: 7.0 + 2.7 + 14.5.
#include "rts_device.hpp"
#include "rts_internal.h"
#include "../../include/row_top_select.h"

namespace rts {

constexpr int kPoolBlock = 1024;
constexpr int kPoolWaves = kPoolBlock / kWave;

// Words of a bit a block, in whole 16 bytes.
__host__ __device__ __forceinline__ int words_of(int32_t pool) { return (pool + 127) / 128 * 4; }

// The exclusive sums of x and y over the workgroup's threads, and the whole sums.
// Once in a kernel: nothing guards wave_sum from a scan before.
struct Sums {
    uint32_t x, y, all_x, all_y;
};
__device__ __forceinline__ Sums block_scan(uint32_t x, uint32_t y, uint2* wave_sum) {
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const uint32_t inc_x = wave_incl_scan32(x), inc_y = wave_incl_scan32(y);
    if (lane == kWave - 1) wave_sum[wave] = uint2{inc_x, inc_y};
    __syncthreads();
    const uint2 of_lane = lane < kPoolWaves ? wave_sum[lane] : uint2{0, 0};
    const uint32_t upto_x = wave_incl_scan32(of_lane.x), upto_y = wave_incl_scan32(of_lane.y);
    const int w = __builtin_amdgcn_readfirstlane(wave);
    Sums s;
    s.x = inc_x - x + (w > 0 ? __builtin_amdgcn_readlane(upto_x, w - 1) : 0);
    s.y = inc_y - y + (w > 0 ? __builtin_amdgcn_readlane(upto_y, w - 1) : 0);
    s.all_x = __builtin_amdgcn_readlane(upto_x, kPoolWaves - 1);
    s.all_y = __builtin_amdgcn_readlane(upto_y, kPoolWaves - 1);
    return s;
}

__device__ __forceinline__ void set_bit(uint32_t* bits, uint32_t i) { atomicOr(&bits[i >> 5], 1u << (i & 31)); }
__device__ __forceinline__ bool get_bit(const uint32_t* bits, uint32_t i) { return bits[i >> 5] >> (i & 31) & 1; }

// Which of four bytes are not 0.
__device__ __forceinline__ uint32_t set_bytes(uint32_t v) {
    const uint32_t high = (((v & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | v) & 0x80808080u;
    return (high >> 7) * 0x10204080u >> 28;
}
// put(w, bits) for words [lo, hi) of `held`, bit b of word w: held[32 w + b] is not 0.
template <typename Put>
__device__ __forceinline__ void held_words(const uint8_t* held, int pool, int lo, int hi, Put&& put) {
    if (!held) return;
    constexpr int kAhead = 4;
    const bool whole = ((uintptr_t)held & 15) == 0;
    for (int w0 = lo + threadIdx.x; w0 < hi; w0 += kPoolBlock * kAhead) {
        uint4 x[kAhead][2] = {};
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int w = w0 + u * kPoolBlock;
            if (whole && w < hi && w * 32 + 32 <= pool) {
                const uint4* p = reinterpret_cast<const uint4*>(held + (int64_t)w * 32);
                x[u][0] = p[0], x[u][1] = p[1];
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int w = w0 + u * kPoolBlock, left = pool - w * 32;
            if (w >= hi) break;
            uint32_t bits = 0;
            if (!whole || left < 32) {
                for (int b = 0; b < 32 && b < left; ++b) bits |= (uint32_t)(held[(int64_t)w * 32 + b] != 0) << b;
            } else {
                const uint32_t v[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
#pragma unroll
                for (int i = 0; i < 8; ++i) bits |= set_bytes(v[i]) << 4 * i;
            }
            put(w, bits);
        }
    }
}
// The same for a workgroup's share of them.
template <typename Put>
__device__ __forceinline__ void held_share(const uint8_t* held, int pool, int words, Put&& put) {
    const int per = (words + gridDim.x - 1) / gridDim.x, lo = blockIdx.x * per;
    held_words(held, pool, lo, lo + per < words ? lo + per : words, put);
}
// Words [0, words) of LDS, 16 bytes at a time.
__device__ __forceinline__ void clear(uint32_t* bits, int words) {
    for (int w = threadIdx.x * 4; w < words; w += kPoolBlock * 4) *reinterpret_cast<uint4*>(bits + w) = uint4{0, 0, 0, 0};
}
__device__ __forceinline__ void store_field(uint32_t* to, const uint32_t* bits, int words) {
    for (int w = threadIdx.x * 4; w < words; w += kPoolBlock * 4)
        *reinterpret_cast<uint4*>(to + w) = *reinterpret_cast<const uint4*>(bits + w);
}
// The bits of word w that are no block's.
__device__ __forceinline__ uint32_t behind(int pool, int w) {
    const int left = pool - w * 32;
    return left >= 32 ? 0 : left <= 0 ? ~0u : ~0u << left;
}

// Four entries of a table row at any address, and what of them lies inside of it.
typedef int ids4 __attribute__((ext_vector_type(4)));
typedef int ids4_at4 __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ ids4 four_entries(const int32_t* row, int j, int n) {
    ids4 x = {-1, -1, -1, -1};
    if (j + 4 <= n)
        x = *reinterpret_cast<const ids4_at4*>(row + j);
    else if (j < n) {
        x[0] = row[j];
        if (j + 1 < n) x[1] = row[j + 1];
        if (j + 2 < n) x[2] = row[j + 2];
    }
    return x;
}

// Sets the bits of the first n(row) entries of rows [lo, hi) of a table.  A wave takes 64 rows' lengths at a time and reads eight rows side by side, 256 entries each.
template <typename Count>
__device__ __forceinline__ void mark_rows(const int32_t* table, int64_t ld, int64_t lo, int64_t hi, int pool,
                                          uint32_t* bits, Count&& n) {
    constexpr int kRows = 8;
    const int lane = lane_id();
    for (int64_t r0 = lo; r0 < hi; r0 += kWave) {
        const int count = r0 + lane < hi ? n(r0 + lane) : 0;
        uint64_t todo = __ballot(count > 0);
        while (todo) {
            int row[kRows], c[kRows], most = 0;
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                row[u] = todo ? __builtin_ctzll(todo) : 0;
                c[u] = todo ? __builtin_amdgcn_readlane(count, row[u]) : 0;
                most = c[u] > most ? c[u] : most;
                todo &= todo - 1;
            }
            for (int j = lane * 4; j - lane * 4 < most; j += 4 * kWave) {
                ids4 id[kRows];
#pragma unroll
                for (int u = 0; u < kRows; ++u) id[u] = four_entries(table + (r0 + row[u]) * ld, j, c[u]);
#pragma unroll
                for (int u = 0; u < kRows; ++u)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if ((uint32_t)id[u][v] < (uint32_t)pool) set_bit(bits, id[u][v]);
            }
        }
    }
}
// A wave's share of rows.
__device__ __forceinline__ void rows_of(int64_t part, int64_t parts, int64_t rows, int64_t& lo, int64_t& hi) {
    const int64_t per = (rows + parts - 1) / parts;
    lo = part * per < rows ? part * per : rows;
    hi = lo + per < rows ? lo + per : rows;
}

// The same of narrow tables, whose rows would leave most of a wave idle: a lane
// takes an entry, eight on their way, of entries [lo, hi) of the table read row by row.
template <typename Count>
__device__ __forceinline__ void mark_entries(const int32_t* table, int64_t ld, uint32_t cols, uint32_t lo, uint32_t hi,
                                             int pool, uint32_t* bits, Count&& n) {
    constexpr int kAhead = 8;
    for (uint32_t e0 = lo + threadIdx.x; e0 < hi; e0 += kAhead * kPoolBlock) {
        int id[kAhead];
        bool inside[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const uint32_t e = e0 + u * kPoolBlock, at = e < hi ? e : lo, r = at / cols, j = at - r * cols;
            id[u] = table[(int64_t)r * ld + j];
            inside[u] = e < hi && (int)j < n(r);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (inside[u] && (uint32_t)id[u] < (uint32_t)pool) set_bit(bits, id[u]);
    }
}
// Rows of a workgroup below which a table is read so too, us by rows and by entries: 6 x 7772 entries 38 and 27,
// 64 x 8192 59 and 26; 16 x 4096 28 and 34.
constexpr int kFew = kPoolWaves;
constexpr int kNarrow = 128;  // columns below which a table is: 1568 rows of 4 columns 122 us by rows, 17 so
template <typename Count>
__device__ __forceinline__ void mark_table(const int32_t* table, int64_t ld, int cols, int64_t rows, int64_t part,
                                           int64_t parts, int pool, uint32_t* bits, Count&& n) {
    if (cols < kNarrow || rows < kFew * parts) {
        const uint32_t all = (uint32_t)rows * (uint32_t)cols, per = (all + (uint32_t)parts - 1) / (uint32_t)parts;
        const uint32_t lo = (uint32_t)part * per < all ? (uint32_t)part * per : all;
        mark_entries(table, ld, cols, lo, lo + per < all ? lo + per : all, pool, bits, n);
    } else {
        int64_t lo, hi;
        rows_of(part * kPoolWaves + threadIdx.x / kWave, parts * kPoolWaves, rows, lo, hi);
        mark_rows(table, ld, lo, hi, pool, bits, n);
    }
}

// Words of LDS bits a thread counts: twice an odd number, so that the lanes'
// 8-byte reads lie in different banks.
__device__ __forceinline__ int unit_of(int words) { return (((words + 2 * kPoolBlock - 1) / (2 * kPoolBlock)) | 1) * 2; }
constexpr int kMaxUnitPairs = ((kMaxPool / 32 + 2 * kPoolBlock - 1) / (2 * kPoolBlock)) | 1;

// The position of the n-th set bit of x, from 0.
__device__ __forceinline__ int nth_bit(uint64_t x, uint32_t n) {
    int at = 0;
#pragma unroll
    for (int w = 32; w > 0; w >>= 1) {
        const uint32_t c = __popcll(x & ((1ull << w) - 1));
        if (n >= c) n -= c, x >>= w, at += w;
    }
    return at;
}

// The block of rank r among the bits of pair(p), the p-th 64 of them, before(u) the
// rank of unit u's first and `pairs` words' pairs a unit.
template <typename Pair, typename Before>
__device__ __forceinline__ int find_rank(uint32_t r, int pairs, int all_pairs, Pair&& pair, Before&& before) {
    int lo = 0, hi = (all_pairs + pairs - 1) / pairs;  // the last unit with at most r bits before it
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before(mid) <= r) lo = mid; else hi = mid;
    }
    r -= before(lo);
    uint64_t bits = 0, x[kMaxUnitPairs];
    const int p0 = lo * pairs;
    int at = p0;
    uint32_t passed = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kMaxUnitPairs; ++i) x[i] = i < pairs && p0 + i < all_pairs ? pair(p0 + i) : 0;
#pragma unroll
    for (int i = 0; i < kMaxUnitPairs; ++i) {
        if (r >= sum) at = p0 + i, bits = x[i], passed = sum;
        sum += __popcll(x[i]);
    }
    return at * 64 + nth_bit(bits, r - passed);
}

// Writes the ids of the bits set in pair(p), ascending, to out[rank - skip] for ranks
// in [skip, skip + n): a wave takes a run of units, four pairs at a time, a lane an id.
template <typename Pair, typename Before>
__device__ __forceinline__ void list_bits(int all_pairs, int pairs, uint32_t part, uint32_t parts, uint32_t skip,
                                          int64_t n, int32_t* out, Pair&& pair, Before&& before) {
    constexpr int kAhead = 4;
    const int lane = lane_id();
    const int units = (all_pairs + pairs - 1) / pairs;
    const int per = (units + parts - 1) / parts;
    const int u0 = part * per, u1 = u0 + per < units ? u0 + per : units;
    if (u0 >= u1) return;
    uint32_t rank = before(u0);
    const int end = u1 * pairs < all_pairs ? u1 * pairs : all_pairs;
    for (int p = u0 * pairs; p < end; p += kAhead) {
        uint64_t x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) x[i] = p + i < end ? pair(p + i) : 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const uint32_t r = rank + mbcnt64(x[i]);
            if ((x[i] >> lane & 1) && r >= skip && (int64_t)(r - skip) < n) out[r - skip] = (p + i) * 64 + lane;
            rank += __popcll(x[i]);
        }
    }
}

struct Lengths {
    int full, need;  // whole blocks, and blocks begun; both within the table
};
__device__ __forceinline__ Lengths lengths(int32_t ctx, int32_t block_size, int32_t cols) {
    const int c = ctx > 0 ? ctx : 0;
    const int full = c / block_size, need = full + (c - full * block_size != 0);
    return {full < cols ? full : cols, need < cols ? need : cols};
}

// Every entry of a table: entry(row, column), kAhead of a thread side by side.
template <int kAhead, typename Entry>
__device__ __forceinline__ void write_table(int32_t* table, int64_t ld, int cols, int64_t rows, int64_t at, int64_t step,
                                            Entry&& entry) {
    const uint32_t all = (uint32_t)rows * (uint32_t)cols;
    for (int64_t e0 = at; e0 < all; e0 += kAhead * step) {
        int32_t id[kAhead], *to[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t e = e0 + u * step;
            const uint32_t i = (uint32_t)(e < all ? e : at) / (uint32_t)cols, j = (uint32_t)(e < all ? e : at) - i * cols;
            to[u] = table + i * ld + j;
            id[u] = entry(i, (int)j);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (e0 + u * step < all) *to[u] = id[u];
    }
}

constexpr int kForkRowsEach = kMaxForkRows / kPoolBlock;  // rows of a thread
constexpr int kNoRow = 0x7FFFFFFF;
// Clears `first` and finds each parent's first row.  Ends behind a barrier.
__device__ __forceinline__ void first_rows(const ForkArgs& a, int* first, const int (&par)[kForkRowsEach]) {
    for (int p = threadIdx.x; p < a.rows_in; p += kPoolBlock) first[p] = kNoRow;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kForkRowsEach; ++u)
        if (par[u] >= 0) atomicMin(&first[par[u]], (int)threadIdx.x * kForkRowsEach + u);
    __syncthreads();
}
// The parents of a thread's neighbouring rows, -1 where there is none.
__device__ __forceinline__ void load_parents(const ForkArgs& a, int (&par)[kForkRowsEach]) {
#pragma unroll
    for (int u = 0; u < kForkRowsEach; ++u) {
        const int i = threadIdx.x * kForkRowsEach + u;
        par[u] = i < a.rows_out ? a.parents[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < kForkRowsEach; ++u)
        if ((uint32_t)par[u] >= (uint32_t)a.rows_in) par[u] = -1;
}

// Where tables are large, the bits of their entries are formed by several
// workgroups, each of a share of the rows and of the held blocks, into bit fields of the whole pool
// that a further launch joins to one.
__global__ __launch_bounds__(kPoolBlock) void mark_fork_kernel(ForkArgs a, uint32_t* __restrict__ fields) {
    extern __shared__ __align__(16) uint32_t lds[];
    const int words = words_of(a.pool);
    uint32_t* const used = lds;
    int* const first = reinterpret_cast<int*>(used + words);
    int par[kForkRowsEach];
    load_parents(a, par);
    clear(used, words);
    first_rows(a, first, par);
    held_share(a.held, a.pool, words, [&](int w, uint32_t bits) { atomicOr(&used[w], bits); });
    mark_table(a.table, a.ld_table, a.cols, a.rows_in, blockIdx.x, gridDim.x, a.pool, used,
               [&](int64_t p) { return first[p] == kNoRow ? 0 : lengths(a.ctx_lens[p], a.block_size, a.cols).full; });
    __syncthreads();
    store_field(fields + (int64_t)blockIdx.x * words, used, words);
}
__global__ __launch_bounds__(kPoolBlock) void mark_compact_kernel(CompactArgs a, uint32_t* __restrict__ fields) {
    extern __shared__ __align__(16) uint32_t lds[];
    const int words = words_of(a.pool);
    clear(lds, words);
    __syncthreads();
    uint32_t* const held = fields + (int64_t)gridDim.x * words;  // a field of their own
    held_share(a.held, a.pool, words, [&](int w, uint32_t bits) { held[w] = bits; });
    mark_table(a.table, a.ld_table, a.cols, a.rows, blockIdx.x, gridDim.x, a.pool, lds,
               [&](int64_t r) { return lengths(a.ctx_lens[r], a.block_size, a.cols).need; });
    __syncthreads();
    store_field(fields + (int64_t)blockIdx.x * words, lds, words);
}
// Field 0 becomes all n fields' bits, four words a thread.
constexpr int kJoinBlock = 64;
__global__ __launch_bounds__(kJoinBlock) void join_fields_kernel(uint32_t* fields, int n, int words) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    constexpr int kAhead = 8;
    const int w = (blockIdx.x * kJoinBlock + threadIdx.x) * 4;
    if (w >= words) return;
    u32x4 bits = {0, 0, 0, 0};
    for (int f = 0; f < n; f += kAhead) {
        u32x4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            x[u] = *reinterpret_cast<const u32x4*>(fields + (int64_t)(f + u < n ? f + u : f) * words + w);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) bits |= x[u];
    }
    *reinterpret_cast<u32x4*>(fields + w) = bits;
}
static int launch_join_fields(uint32_t* fields, int n, int words, hipStream_t s) {
    hipLaunchKernelGGL(join_fields_kernel, dim3((unsigned)(words / 4 + kJoinBlock - 1) / kJoinBlock), dim3(kJoinBlock), 0, s,
                       fields, n, words);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}
// dst = a field, four loads of 16 bytes of a thread on their way.
__device__ __forceinline__ void load_field(const uint32_t* field, int words, uint32_t* dst) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    constexpr int kAhead = 4;
    for (int w0 = threadIdx.x * 4; w0 < words; w0 += kPoolBlock * 4 * kAhead) {
        u32x4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int w = w0 + u * kPoolBlock * 4;
            x[u] = *reinterpret_cast<const u32x4*>(field + (w < words ? w : w0));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int w = w0 + u * kPoolBlock * 4;
            if (w < words) *reinterpret_cast<u32x4*>(dst + w) = x[u];
        }
    }
}

__global__ __launch_bounds__(kPoolBlock) void fork_blocks_kernel(ForkArgs a, const uint32_t* __restrict__ field) {
    extern __shared__ __align__(16) uint32_t lds[];
    __shared__ uint2 wave_sum[kPoolWaves];
    __shared__ uint32_t free_before[kPoolBlock];
    const int words = words_of(a.pool);
    const int rows_in = (int)a.rows_in, rows = (int)a.rows_out;
    uint32_t* const used = lds;                                      // a bit a block
    uint32_t* const twice = used + words;                            // last blocks that no row may keep
    int* const got = reinterpret_cast<int*>(twice);                  // afterwards: a row's fresh block
    int* const first = reinterpret_cast<int*>(twice + (words > rows ? words : rows));  // a parent's first row
    int* const fresh = first;                                        // afterwards: the fresh blocks
    const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;

    // Every parent's last block, where it is being written, beside the rest.
    int par[kForkRowsEach], ctx[kForkRowsEach], last[kForkRowsEach];
    load_parents(a, par);
#pragma unroll
    for (int u = 0; u < kForkRowsEach; ++u) {
        const int p = tid + u * kPoolBlock;
        ctx[u] = p < rows_in ? a.ctx_lens[p] : 0;
    }
#pragma unroll
    for (int u = 0; u < kForkRowsEach; ++u) {
        const Lengths n = lengths(ctx[u], a.block_size, a.cols);
        last[u] = n.full < n.need ? a.table[(tid + u * kPoolBlock) * a.ld_table + n.full] : -1;
        if ((uint32_t)last[u] >= (uint32_t)a.pool) last[u] = -1;
    }
    if (field) clear(twice, words);
    else clear(used, 2 * words);
    if (field) load_field(field, words, used);
    first_rows(a, first, par);
    if (!field)
        held_words(a.held, a.pool, 0, words, [&](int w, uint32_t bits) { atomicOr(&used[w], bits); });
    __syncthreads();
    if (tid < 4 && words > 0) atomicOr(&used[words - 4 + tid], behind(a.pool, words - 4 + tid));
    if (!field) {
        mark_table(a.table, a.ld_table, a.cols, rows_in, 0, 1, a.pool, used, [&](int64_t p) {
            return first[p] == kNoRow ? 0 : lengths(a.ctx_lens[p], a.block_size, a.cols).full;
        });
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kForkRowsEach; ++u) {
        const int p = tid + u * kPoolBlock;
        if (p >= rows_in || first[p] == kNoRow) continue;
        const uint32_t id = last[u];
        if (last[u] >= 0) {
            const uint32_t bit = 1u << (id & 31);
            if (atomicOr(&used[id >> 5], bit) & bit) atomicOr(&twice[id >> 5], bit);
        }
        // Its first row and its last block in one word.
        static_assert(kMaxForkRows <= 1 << 12 && kMaxPool <= 1 << 19, "31 bits");
        first[p] = last[u] < 0 ? -1 : (int)(id | (uint32_t)first[p] << 19);
    }
    __syncthreads();

    // The rows that want a fresh block, neighbouring ones a thread.
    uint32_t own = 0;
#pragma unroll
    for (int u = 0; u < kForkRowsEach; ++u) {
        const int i = tid * kForkRowsEach + u;
        last[u] = -1;  // from here on: the block to copy
        const int x = par[u] >= 0 ? first[par[u]] : -1;
        if (x < 0) continue;
        const int id = x & ((1 << 19) - 1);
        if (x >> 19 == i && !get_bit(twice, id)) continue;
        last[u] = id;
        ++own;
    }
    // Free blocks in each thread's words.
    const int pairs = unit_of(words) / 2;
    const uint64_t* const used2 = reinterpret_cast<const uint64_t*>(used);
    auto free_pair = [&](int p) { return ~used2[p]; };
    uint32_t mine = 0;
    for (int p = tid * pairs; p < (tid + 1) * pairs && p < words / 2; ++p) mine += __popcll(free_pair(p));
    const Sums sums = block_scan(own, mine, wave_sum);
    const uint32_t wanted = sums.all_x, all_free = sums.all_y;
    uint32_t rank = sums.x;
    free_before[tid] = sums.y;
    __syncthreads();
    auto before = [&](int u) { return free_before[u]; };
    // The lowest of them for the rows that want one, a unit a wave.
    for (int u = wave; u * pairs < words / 2 && free_before[u] < wanted; u += kPoolWaves) {
        uint32_t r = free_before[u];
        for (int p = u * pairs; p < (u + 1) * pairs && p < words / 2; ++p) {
            const uint64_t x = free_pair(p);
            const uint32_t mine = r + mbcnt64(x);
            if ((x >> lane & 1) && mine < wanted) fresh[mine] = p * 64 + lane;
            r += __popcll(x);
        }
    }
    __syncthreads();
    const uint32_t taken = wanted < all_free ? wanted : all_free;
    const bool lead = blockIdx.x == 0;
#pragma unroll
    for (int u = 0; u < kForkRowsEach; ++u) {
        const int i = tid * kForkRowsEach + u;
        if (i >= rows) break;
        got[i] = -2;  // keeps what its parent has
        if (last[u] < 0) continue;
        got[i] = rank < taken ? fresh[rank] : -1;
        if (lead && rank < taken) reinterpret_cast<int2*>(a.copies)[rank] = int2{last[u], fresh[rank]};
        ++rank;
    }
    __syncthreads();

    const int64_t at = (int64_t)blockIdx.x * kPoolBlock + tid, step = (int64_t)gridDim.x * kPoolBlock;
    const uint32_t part = blockIdx.x * kPoolWaves + wave, parts = gridDim.x * kPoolWaves;
    if (at == 0) a.counts[0] = (int32_t)(all_free - taken), a.counts[1] = (int32_t)wanted;
    for (int64_t r = taken + at; r < rows; r += step) reinterpret_cast<int2*>(a.copies)[r] = int2{-1, -1};
    for (int64_t r = (int64_t)(all_free - taken) + at; r < a.n_free; r += step) a.free_blocks[r] = -1;
    list_bits(words / 2, pairs, part, parts, taken, a.n_free, a.free_blocks, free_pair, before);
    for (int i = at; i < rows; i += step) {
        const uint32_t p = a.parents[i];
        const int len = p < (uint32_t)rows_in ? a.ctx_lens[p] : 0;
        a.out_ctx[i] = len > 0 ? len : 0;
    }
    write_table<4>(a.out_table, a.ld_out, a.cols, rows, at, step, [&](uint32_t i, int j) {
        const uint32_t p = a.parents[i];
        if (p >= (uint32_t)rows_in) return -1;
        const int len = a.ctx_lens[p], id = a.table[(int64_t)p * a.ld_table + j], own_block = got[i];
        const Lengths n = lengths(len, a.block_size, a.cols);
        if (j >= n.need || (uint32_t)id >= (uint32_t)a.pool) return j == n.full && own_block != -2 ? own_block : -1;
        return j == n.full && own_block != -2 ? own_block : id;
    });
}

// Bit fields of large tables, one for 16384 entries (for 8192 nothing is gained): none where
// every workgroup reads the table itself in about the time of two more launches.  Calls of
// fork_blocks and compact_blocks, us, without fields: 160 x 257 entries 15 and 15, 320 x 257
// 20 and 21, 512 x 257 23 and 27, 800 x 513 46 and 64; with them 19 and 18, 19 and 18, 19 and 19, 25 and 30.
static int mark_parts(int64_t rows, int32_t cols) {
    const int64_t entries = rows * (int64_t)cols;
    return entries <= 81920 ? 0 : entries < 32 * 16384 ? (int)((entries + 16383) / 16384) : 32;
}
size_t fork_blocks_bytes(int64_t rows, int32_t cols, int32_t pool) {
    return (size_t)mark_parts(rows, cols) * words_of(pool) * 4;
}

static int64_t pool_grid(int64_t work) { return work / 2048 < 1 ? 1 : work / 2048 < 256 ? work / 2048 : 256; }

int launch_fork_blocks(const ForkArgs& a, void* workspace, hipStream_t s) {
    const size_t words = words_of(a.pool);
    const int parts = workspace && words ? mark_parts(a.rows_in, a.cols) : 0;
    uint32_t* fields = static_cast<uint32_t*>(workspace);
    if (parts) {
        hipLaunchKernelGGL(mark_fork_kernel, dim3(parts), dim3(kPoolBlock), (words + a.rows_in) * 4, s, a, fields);
        if (hipGetLastError() != hipSuccess || launch_join_fields(fields, parts, (int)words, s)) return RTS_EHIP;
    }
    const size_t rows = a.rows_out, most = a.rows_in > a.rows_out ? a.rows_in : a.rows_out;
    hipLaunchKernelGGL(fork_blocks_kernel, dim3((unsigned)pool_grid(a.rows_out * (int64_t)a.cols + a.n_free)),
                       dim3(kPoolBlock), (words + (words > rows ? words : rows) + most) * 4, s, a, parts ? fields : nullptr);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

// Compaction.  With n live blocks that may move (those not held), let T be the
// smallest bound below which there are n blocks that are not held.  Live ones at
// or past T move, in ascending order, to the free ones below it: there are as
// many of one as of the other, and no block is both left and taken.
__global__ __launch_bounds__(kPoolBlock) void compact_blocks_kernel(CompactArgs a, const uint32_t* __restrict__ field,
                                                                    const uint32_t* __restrict__ held) {
    extern __shared__ __align__(16) uint32_t lds[];
    __shared__ uint2 wave_sum[kPoolWaves];
    __shared__ uint32_t open_before[kPoolBlock];  // blocks that are not held
    __shared__ uint32_t live_before[kPoolBlock];  // of those, live ones
    __shared__ uint32_t limit[2];                 // T, and the live ones below it
    const int words = words_of(a.pool);
    uint32_t* const live = lds;           // not held, in a table
    uint32_t* const open = live + words;  // not held
    const uint64_t *const live2 = reinterpret_cast<const uint64_t*>(live), *const open2 = reinterpret_cast<const uint64_t*>(open);
    const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
    if (field) {
        load_field(field, words, live);
        if (held) load_field(held, words, open);
        else clear(open, words);
        __syncthreads();
    } else {
        clear(live, 2 * words);
        __syncthreads();
        held_words(a.held, a.pool, 0, words, [&](int w, uint32_t bits) { atomicOr(&open[w], bits); });
        mark_table(a.table, a.ld_table, a.cols, a.rows, 0, 1, a.pool, live,
                   [&](int64_t r) { return lengths(a.ctx_lens[r], a.block_size, a.cols).need; });
        __syncthreads();
    }
    if (tid < 4 && words > 0) open[words - 4 + tid] |= behind(a.pool, words - 4 + tid);
    __syncthreads();
    const int all_pairs = words / 2, pairs = unit_of(words) / 2;
    const int p0 = tid * pairs < all_pairs ? tid * pairs : all_pairs, p1 = p0 + pairs < all_pairs ? p0 + pairs : all_pairs;
    uint32_t n_open = 0, n_live = 0;
    for (int p = p0; p < p1; ++p) {
        const uint64_t o = ~open2[p], l = live2[p] & o;  // held until here
        reinterpret_cast<uint64_t*>(open)[p] = o;
        reinterpret_cast<uint64_t*>(live)[p] = l;
        n_open += __popcll(o);
        n_live += __popcll(l);
    }
    const Sums sums = block_scan(n_open, n_live, wave_sum);
    const uint32_t all_open = sums.all_x, all_live = sums.all_y, before_open = sums.x, before_live = sums.y;
    open_before[tid] = before_open;
    live_before[tid] = before_live;
    if (tid == 0 && all_live == 0) limit[0] = limit[1] = 0;
    if (before_open < all_live && before_open + n_open >= all_live) {  // the n-th open block is among this thread's
        uint32_t o = before_open, l = before_live;
        for (int p = p0; p < p1; ++p) {
            const uint32_t c = __popcll(open2[p]);
            if (o + c >= all_live) {
                const int b = nth_bit(open2[p], all_live - o - 1);
                limit[0] = p * 64 + b + 1;
                limit[1] = l + __popcll(live2[p] & (~0ull >> (63 - b)));
                break;
            }
            o += c;
            l += __popcll(live2[p]);
        }
    }
    __syncthreads();
    const uint32_t bound = limit[0], below = limit[1], wanted = all_live - below;
    const uint32_t moved = (int64_t)wanted < a.max_moves ? wanted : (uint32_t)a.max_moves;

    // Bits of pair p at or past the bound.
    auto past = [&](int p) {
        const int d = (int)bound - p * 64;
        return d <= 0 ? ~0ull : d >= 64 ? 0ull : ~0ull << d;
    };
    // The live blocks before block b.
    auto live_rank = [&](uint32_t b) {
        const int p = b >> 6, u = p / pairs, q = u * pairs;
        uint32_t r = live_before[u];
#pragma unroll
        for (int i = 0; i < kMaxUnitPairs; ++i) r += q + i < p ? __popcll(live2[q + i]) : 0;
        return r + __popcll(live2[p] & ~(~0ull << (b & 63)));
    };
    // The r-th free block (r below `wanted`: it lies below the bound).
    auto free_block = [&](uint32_t r) {
        return find_rank(r, pairs, all_pairs, [&](int p) { return open2[p] & ~live2[p]; },
                         [&](int u) { return open_before[u] - live_before[u]; });
    };

    const int64_t at = (int64_t)blockIdx.x * kPoolBlock + tid, step = (int64_t)gridDim.x * kPoolBlock;
    const uint32_t part = blockIdx.x * kPoolWaves + wave, parts = gridDim.x * kPoolWaves;
    const uint32_t all_free = all_open - all_live;
    if (at == 0) a.counts[0] = (int32_t)all_free, a.counts[1] = (int32_t)wanted;
    for (int64_t r = moved + at; r < a.max_moves; r += step) reinterpret_cast<int2*>(a.moves)[r] = int2{-1, -1};
    for (int64_t r = all_free + at; r < a.n_free; r += step) a.free_blocks[r] = -1;
    // Moves: sources by their rank past the bound, destinations by theirs below.
    {
        const int units = (all_pairs + pairs - 1) / pairs, per = (units + parts - 1) / parts;
        const int u0 = part * per, u1 = u0 + per < units ? u0 + per : units;
        if (u0 < u1) {
            uint32_t o = open_before[u0], l = live_before[u0];
            const int e = u1 * pairs < all_pairs ? u1 * pairs : all_pairs;
            for (int p = u0 * pairs; p < e; ++p) {
                const uint64_t ob = open2[p], lb = live2[p], pb = past(p);
                const uint32_t lr = l + mbcnt64(lb), fr = o + mbcnt64(ob) - lr;  // live and free ones before this lane's
                const bool is_open = ob >> lane & 1, is_live = lb >> lane & 1, is_past = pb >> lane & 1;
                const int id = p * 64 + lane;
                if (is_live && is_past && lr - below < moved) a.moves[2 * (int64_t)(lr - below)] = id;
                if (is_open && !is_live && !is_past && fr < moved) a.moves[2 * (int64_t)fr + 1] = id;
                // Free afterwards: what was free and is not taken, and what was left.
                int64_t rank = -1;
                if (is_open && !is_past) {
                    if (!is_live && fr >= moved) rank = fr - moved;
                } else if (is_open) {
                    const uint32_t left = lr - below < moved ? lr - below : moved;  // sources before this block
                    if (!is_live || lr - below < moved) rank = (int64_t)fr - moved + left;
                }
                if (rank >= 0 && rank < a.n_free) a.free_blocks[rank] = id;
                o += __popcll(ob);
                l += __popcll(lb);
            }
        }
    }
    // A lookup takes some hundred cycles, so there are threads for an entry each, up to the chip's.
    write_table<1>(a.out_table, a.ld_out, a.cols, a.rows, at, step, [&](uint32_t i, int j) {
        const int id = a.table[i * a.ld_table + j];
        if (j >= lengths(a.ctx_lens[i], a.block_size, a.cols).need || (uint32_t)id >= (uint32_t)a.pool) return -1;
        if ((uint32_t)id >= bound && get_bit(live, id)) {
            const uint32_t k = live_rank(id) - below;
            if (k < moved) return free_block(k);
        }
        return id;
    });
}

size_t compact_blocks_bytes(int64_t rows, int32_t cols, int32_t pool) {
    const int parts = mark_parts(rows, cols);
    return parts ? (size_t)(parts + 1) * words_of(pool) * 4 : 0;  // one for the held blocks
}

int launch_compact_blocks(const CompactArgs& a, void* workspace, hipStream_t s) {
    const size_t words = words_of(a.pool);
    const int parts = workspace && words ? mark_parts(a.rows, a.cols) : 0;
    uint32_t* fields = static_cast<uint32_t*>(workspace);
    if (parts) {
        hipLaunchKernelGGL(mark_compact_kernel, dim3(parts), dim3(kPoolBlock), words * 4, s, a, fields);
        if (hipGetLastError() != hipSuccess || launch_join_fields(fields, parts, (int)words, s)) return RTS_EHIP;
    }
    const int64_t grid = pool_grid(2 * a.rows * (int64_t)a.cols + a.n_free + 2 * a.max_moves);
    hipLaunchKernelGGL(compact_blocks_kernel, dim3((unsigned)grid), dim3(kPoolBlock), words * 8, s, a,
                       parts ? fields : nullptr, parts && a.held ? fields + (size_t)parts * words : nullptr);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

// Block copies.  A workgroup takes 16 KB (kCopySlice) of a pair's block in one
// cache: four loads a thread, then four stores.  8000 pairs of 45 KB: 150 us (4.8 TB/s
// read and written, as a large copy reaches); 192 pairs of 64 KB 6.3 us.
constexpr int kCopyBlock = 256;  // 1 << 8, as launch_copy_blocks counts
constexpr int kCopyEach = 4;
constexpr int kCopySlice = kCopyBlock * kCopyEach * 16;

typedef uint32_t words4 __attribute__((ext_vector_type(4)));

// Words [first, last) of the block, row_words of them a row of ld bytes, by `lanes`
// threads, of which this is the t-th.
template <typename T>
__device__ __forceinline__ void copy_words(const char* src, char* dst, int64_t ld, int64_t row_words, int64_t first,
                                           int64_t last, int t, int lanes) {
    // Whole slices of rows that follow each other.
    if (last <= row_words && last - first == kCopyBlock * kCopyEach) {
        const int64_t at = (first + t) * (int64_t)sizeof(T);
        T v[kCopyEach];
#pragma unroll
        for (int u = 0; u < kCopyEach; ++u) v[u] = *reinterpret_cast<const T*>(src + at + u * kCopyBlock * (int64_t)sizeof(T));
#pragma unroll
        for (int u = 0; u < kCopyEach; ++u) *reinterpret_cast<T*>(dst + at + u * kCopyBlock * (int64_t)sizeof(T)) = v[u];
        return;
    }
    for (int64_t i = first + t; i < last; i += lanes) {
        const int64_t row = last <= row_words ? 0 : i / row_words, at = row * ld + (i - row * row_words) * (int64_t)sizeof(T);
        *reinterpret_cast<T*>(dst + at) = *reinterpret_cast<const T*>(src + at);
    }
}

// blockIdx.x: pairs, blockIdx.y: slices of all caches' blocks, both in turn.  Where a
// block has fewer words than the workgroup threads, several pairs are copied side
// by side (19542 pairs of blocks of 1584 and 240 bytes: 29 us one by one, 16 so).
// CACHES: how many the arguments have room for (a few hundred bytes of
// arguments are read sooner than a few thousand).
template <int CACHES>
__global__ __launch_bounds__(kCopyBlock) void copy_blocks_kernel(CopyArgs<CACHES> a) {
    for (int64_t s = blockIdx.y; s < a.slices; s += gridDim.y) {
        int c = 0;
        while (c + 1 < a.n_caches && s >= a.cache[c + 1].slice0) ++c;
        const CopyCache k = a.cache[c];
        const int64_t per = kCopySlice / k.word, first = (s - k.slice0) * per;
        const int64_t last = first + per < k.words ? first + per : k.words;
        const int lanes = 1 << k.lanes_log2, beside = kCopyBlock >> k.lanes_log2, t = threadIdx.x & (lanes - 1);
        for (int64_t pair = (int64_t)blockIdx.x * beside + (threadIdx.x >> k.lanes_log2); pair < a.n_pairs;
             pair += (int64_t)gridDim.x * beside) {
            const int2 p = reinterpret_cast<const int2*>(a.pairs)[pair];
            if (p.x < 0 || p.y < 0 || p.x == p.y) continue;
            const int64_t from = p.x * a.stride_rows, to = p.y * a.stride_rows;
            if (from > k.rows - a.block_size || to > k.rows - a.block_size) continue;
            const char* src = k.data + from * k.ld;
            char* dst = k.data + to * k.ld;
            if (k.word == 16) copy_words<words4>(src, dst, k.ld, k.row_words, first, last, t, lanes);
            else if (k.word == 4) copy_words<uint32_t>(src, dst, k.ld, k.row_words, first, last, t, lanes);
            else if (k.word == 2) copy_words<uint16_t>(src, dst, k.ld, k.row_words, first, last, t, lanes);
            else copy_words<uint8_t>(src, dst, k.ld, k.row_words, first, last, t, lanes);
        }
    }
}

template <int CACHES>
static int launch_copy(const CopyArgs<kMaxCopyCaches>& all, hipStream_t s) {
    CopyArgs<CACHES> a;
    a.pairs = all.pairs, a.n_pairs = all.n_pairs, a.stride_rows = all.stride_rows, a.slices = all.slices;
    a.n_caches = all.n_caches, a.block_size = all.block_size;
    for (int c = 0; c < all.n_caches; ++c) a.cache[c] = all.cache[c];
    int widest = 0;
    for (int c = 0; c < all.n_caches; ++c) widest = a.cache[c].lanes_log2 > widest ? a.cache[c].lanes_log2 : widest;
    const int64_t beside = kCopyBlock >> widest, units = (a.n_pairs + beside - 1) / beside;
    const unsigned y = a.slices < 4096 ? (unsigned)a.slices : 4096, most = 8192 / y > 1 ? 8192 / y : 1;
    const unsigned x = units < most ? (unsigned)units : most;
    hipLaunchKernelGGL(copy_blocks_kernel<CACHES>, dim3(x, y), dim3(kCopyBlock), 0, s, a);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

int launch_copy_blocks(CopyArgs<kMaxCopyCaches>& a, hipStream_t s) {
    a.slices = 0;
    for (int c = 0; c < a.n_caches; ++c) {
        CopyCache& k = a.cache[c];
        k.slice0 = a.slices;
        a.slices += (k.words * k.word + kCopySlice - 1) / kCopySlice;
        for (k.lanes_log2 = 8; k.lanes_log2 > 3 && 1 << (k.lanes_log2 - 1) >= k.words; --k.lanes_log2) {}
    }
    return a.n_caches <= 4 ? launch_copy<4>(a, s) : launch_copy<kMaxCopyCaches>(a, s);
}

}  // namespace rts
