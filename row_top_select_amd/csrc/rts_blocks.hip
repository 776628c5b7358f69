// Forking, freeing, compacting and copying the blocks of a paged cache, for
// gfx950.
//
// Which blocks are in use is not kept anywhere: it follows from the block
// tables and lengths, one bit a block.  Every workgroup forms these bits for
// the whole pool by itself in LDS (64 KB for 2^19 blocks), takes the ranks that
// it needs from them and writes its share of the outputs, so that no workgroup
// reads what another one writes and one launch does all of it.  The work is a
// few bytes a block and table entry: what counts is latency.
#include "rts_device.hpp"
#include "rts_internal.h"
#include "../../include/row_top_select.h"

namespace rts {

constexpr int kPoolBlock = 1024;
constexpr int kPoolWaves = kPoolBlock / kWave;

// The exclusive sum of x over the workgroup's threads; total: the whole sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* wave_sum, uint32_t& total) {
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const uint32_t inc = wave_incl_scan32(x);
    __syncthreads();  // wave_sum may still be read from the scan before
    if (lane == kWave - 1) wave_sum[wave] = inc;
    __syncthreads();
    const uint32_t mine = lane < kPoolWaves ? wave_sum[lane] : 0;
    const uint32_t upto = wave_incl_scan32(mine);
    total = __builtin_amdgcn_readlane(upto, kPoolWaves - 1);
    const uint32_t before = wave > 0 ? __builtin_amdgcn_readlane(upto, wave - 1) : 0;
    return before + inc - x;
}

__device__ __forceinline__ void set_bit(uint32_t* bits, uint32_t i) { atomicOr(&bits[i >> 5], 1u << (i & 31)); }
__device__ __forceinline__ bool get_bit(const uint32_t* bits, uint32_t i) { return bits[i >> 5] >> (i & 31) & 1; }

// Bit b of word w: held[32 w + b] is set, or the pool has no such block and `past` is set.
__device__ __forceinline__ uint32_t held_word(const uint8_t* held, int pool, int w, bool past) {
    const int left = pool - w * 32;
    uint32_t bits = 0;
    if (held) {
        if (left >= 32 && ((uintptr_t)held & 15) == 0) {
            const uint4* p = reinterpret_cast<const uint4*>(held + (int64_t)w * 32);
            const uint4 x[2] = {p[0], p[1]};
            const uint32_t v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int b = 0; b < 4; ++b) bits |= (uint32_t)((v[i] >> (8 * b) & 0xFF) != 0) << (4 * i + b);
        } else
            for (int b = 0; b < 32 && b < left; ++b) bits |= (uint32_t)(held[(int64_t)w * 32 + b] != 0) << b;
    }
    if (past && left < 32) bits |= left <= 0 ? ~0u : ~0u << left;
    return bits;
}

// Sets the bits of the first n(row) entries of each row of a table.  A wave
// takes 64 rows' lengths at a time and reads four rows' entries side by side.
template <typename Count>
__device__ __forceinline__ void mark_rows(const int32_t* table, int64_t ld, int64_t rows, int pool, uint32_t* bits,
                                          Count&& n) {
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int64_t per = (rows + kPoolWaves - 1) / kPoolWaves;
    const int64_t lo = wave * per, hi = lo + per < rows ? lo + per : rows;
    for (int64_t r0 = lo; r0 < hi; r0 += kWave) {
        const int count = r0 + lane < hi ? n(r0 + lane) : 0;
        const int here = (int)(hi - r0 < kWave ? hi - r0 : kWave);
        for (int r = 0; r < here; r += 4) {
            int c[4], most = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                c[u] = r + u < here ? __builtin_amdgcn_readlane(count, r + u) : 0;
                most = c[u] > most ? c[u] : most;
            }
            for (int j0 = 0; j0 < most; j0 += 2 * kWave) {
                int id[4][2];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int j = j0 + v * kWave + lane;
                        id[u][v] = j < c[u] ? table[(r0 + r + u) * ld + j] : -1;
                    }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        if ((uint32_t)id[u][v] < (uint32_t)pool) set_bit(bits, id[u][v]);
            }
        }
    }
}

// The position of the n-th set bit of x, from 0.
__device__ __forceinline__ int nth_bit(uint32_t x, uint32_t n) {
    for (; n > 0; --n) x &= x - 1;
    return __builtin_ctz(x);
}

// Writes the ids of bits set in word(w), ascending, to out[rank - skip] for
// ranks in [skip, skip + n): a wave takes a run of words, two at a time, a lane
// an id.  before(w): the rank of word w's first.  `part` of `parts` waves.
template <typename Word, typename Before>
__device__ __forceinline__ void list_bits(int words, int unit, uint32_t part, uint32_t parts, uint32_t skip, int64_t n,
                                          int32_t* out, Word&& word, Before&& before) {
    const int lane = lane_id();
    const int units = (words + unit - 1) / unit;
    const int per = (units + parts - 1) / parts;
    const int u0 = part * per, u1 = u0 + per < units ? u0 + per : units;
    if (u0 >= u1) return;
    uint32_t rank = before(u0);
    const int w1 = u1 * unit < words ? u1 * unit : words;
    for (int w = u0 * unit; w < w1; w += 2) {
        const uint32_t lo = word(w), hi = w + 1 < w1 ? word(w + 1) : 0;
        const uint64_t both = (uint64_t)hi << 32 | lo;
        const uint32_t r = rank + mbcnt64(both);
        if ((both >> lane & 1) && r >= skip && (int64_t)(r - skip) < n) out[r - skip] = w * 32 + lane;
        rank += __popcll(both);
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

__global__ __launch_bounds__(kPoolBlock) void fork_blocks_kernel(ForkArgs a) {
    extern __shared__ uint32_t lds[];
    __shared__ uint32_t wave_sum[kPoolWaves];
    __shared__ uint32_t free_before[kPoolBlock];
    const int words = (a.pool + 31) / 32;
    const int rows_in = (int)a.rows_in, rows = (int)a.rows_out;
    uint32_t* const used = lds;                                      // a bit a block
    uint32_t* const twice = used + words;                            // last blocks that no row may keep
    int* const got = reinterpret_cast<int*>(twice);                  // afterwards: a row's fresh block
    int* const first = reinterpret_cast<int*>(twice + (words > rows ? words : rows));  // a parent's first row
    int* const fresh = first;                                        // afterwards: the fresh blocks
    const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;

    for (int w = tid; w < words; w += kPoolBlock) {
        used[w] = held_word(a.held, a.pool, w, true);
        twice[w] = 0;
    }
    for (int p = tid; p < rows_in; p += kPoolBlock) first[p] = 0x7FFFFFFF;
    __syncthreads();
    auto parent = [&](int i) {
        const int p = a.parents[i];
        return (uint32_t)p < (uint32_t)rows_in ? p : -1;
    };
    for (int i = tid; i < rows; i += kPoolBlock) {
        const int p = parent(i);
        if (p >= 0) atomicMin(&first[p], i);
    }
    __syncthreads();
    auto shape = [&](int p) { return lengths(a.ctx_lens[p], a.block_size, a.cols); };
    mark_rows(a.table, a.ld_table, rows_in, a.pool, used,
              [&](int64_t p) { return first[p] == 0x7FFFFFFF ? 0 : shape((int)p).full; });
    __syncthreads();
    for (int p = tid; p < rows_in; p += kPoolBlock) {
        if (first[p] == 0x7FFFFFFF) continue;
        const Lengths n = shape(p);
        if (n.full >= n.need) continue;
        const uint32_t id = a.table[p * a.ld_table + n.full];
        if (id >= (uint32_t)a.pool) continue;
        const uint32_t bit = 1u << (id & 31);
        if (atomicOr(&used[id >> 5], bit) & bit) atomicOr(&twice[id >> 5], bit);
    }
    __syncthreads();

    // The rows that want a fresh block, four neighbouring ones a thread.
    constexpr int kRows = kMaxForkRows / kPoolBlock;
    int last[kRows];  // the block to copy, or -1
    uint32_t own = 0;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int i = tid * kRows + u;
        last[u] = -1;
        const int p = i < rows ? parent(i) : -1;
        if (p < 0) continue;
        const Lengths n = shape(p);
        if (n.full >= n.need) continue;
        const uint32_t id = a.table[p * a.ld_table + n.full];
        if (id >= (uint32_t)a.pool || (first[p] == i && !get_bit(twice, id))) continue;
        last[u] = (int)id;
        ++own;
    }
    uint32_t wanted, all_free;
    uint32_t rank = block_scan(own, wave_sum, wanted);
    // Free blocks before each thread's words.
    const int unit = ((words + kPoolBlock - 1) / kPoolBlock + 1) & ~1;  // words a thread, even
    uint32_t mine = 0;
    for (int w = tid * unit; w < (tid + 1) * unit && w < words; ++w) mine += __popc(~used[w]);
    uint32_t before = block_scan(mine, wave_sum, all_free);
    free_before[tid] = before;
    for (int w = tid * unit; w < (tid + 1) * unit && w < words && before < wanted; ++w)
        for (uint32_t x = ~used[w]; x && before < wanted; x &= x - 1) fresh[before++] = w * 32 + __builtin_ctz(x);
    __syncthreads();
    const uint32_t taken = wanted < all_free ? wanted : all_free;
    const bool lead = blockIdx.x == 0;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int i = tid * kRows + u;
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
    list_bits(words, unit, part, parts, taken, a.n_free, a.free_blocks, [&](int w) { return ~used[w]; },
              [&](int u) { return free_before[u]; });
    for (int i = part; i < rows; i += parts) {
        const int p = parent(i);
        int32_t* const out = a.out_table + i * a.ld_out;
        const int ctx = p < 0 ? 0 : a.ctx_lens[p];
        const Lengths n = lengths(ctx, a.block_size, a.cols);
        if (lane == 0) a.out_ctx[i] = ctx > 0 ? ctx : 0;
        const int own_block = got[i];
        for (int j = lane; j < a.cols; j += kWave) {
            int id = -1;
            if (j < n.need) id = a.table[p * a.ld_table + j];
            if ((uint32_t)id >= (uint32_t)a.pool) id = -1;
            if (j == n.full && own_block != -2) id = own_block;
            out[j] = id;
        }
    }
}

int launch_fork_blocks(const ForkArgs& a, hipStream_t s) {
    const int64_t work = a.rows_out * (int64_t)a.cols + a.n_free;
    const int64_t grid = work / 16384 < 1 ? 1 : work / 16384 < 64 ? work / 16384 : 64;
    const int64_t words = (a.pool + 31) / 32;
    const size_t lds = (size_t)(words + (words > a.rows_out ? words : a.rows_out) +
                                (a.rows_in > a.rows_out ? a.rows_in : a.rows_out)) * 4;
    hipLaunchKernelGGL(fork_blocks_kernel, dim3((unsigned)grid), dim3(kPoolBlock), lds, s, a);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

// Compaction.  With n live blocks that may move (those not held), let T be the
// smallest bound below which there are n blocks that are not held.  Live ones at
// or past T move, in ascending order, to the free ones below it: there are as
// many of one as of the other, and no block is both left and taken.
__global__ __launch_bounds__(kPoolBlock) void compact_blocks_kernel(CompactArgs a) {
    extern __shared__ uint32_t lds[];
    __shared__ uint32_t wave_sum[kPoolWaves];
    __shared__ uint32_t open_before[kPoolBlock];  // blocks that are not held
    __shared__ uint32_t live_before[kPoolBlock];  // of those, live ones
    __shared__ uint32_t limit[2];                 // T, and the live ones below it
    const int words = (a.pool + 31) / 32;
    uint32_t* const live = lds;           // not held, in a table
    uint32_t* const open = live + words;  // not held
    const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
    for (int w = tid; w < words; w += kPoolBlock) {
        live[w] = 0;
        open[w] = ~held_word(a.held, a.pool, w, true);
    }
    __syncthreads();
    mark_rows(a.table, a.ld_table, a.rows, a.pool, live,
              [&](int64_t r) { return lengths(a.ctx_lens[r], a.block_size, a.cols).need; });
    __syncthreads();
    const int unit = ((words + kPoolBlock - 1) / kPoolBlock + 1) & ~1;
    const int w0 = tid * unit < words ? tid * unit : words, w1 = w0 + unit < words ? w0 + unit : words;
    uint32_t n_open = 0, n_live = 0;
    for (int w = w0; w < w1; ++w) {
        live[w] &= open[w];
        n_open += __popc(open[w]);
        n_live += __popc(live[w]);
    }
    uint32_t all_open, all_live;
    const uint32_t before_open = block_scan(n_open, wave_sum, all_open);
    const uint32_t before_live = block_scan(n_live, wave_sum, all_live);
    open_before[tid] = before_open;
    live_before[tid] = before_live;
    if (tid == 0 && all_live == 0) limit[0] = limit[1] = 0;
    if (before_open < all_live && before_open + n_open >= all_live) {  // the n-th open block is among this thread's
        uint32_t o = before_open, l = before_live;
        for (int w = w0; w < w1; ++w) {
            const uint32_t c = __popc(open[w]);
            if (o + c >= all_live) {
                const int b = nth_bit(open[w], all_live - o - 1);
                limit[0] = w * 32 + b + 1;
                limit[1] = l + __popc(live[w] & (~0u >> (31 - b)));
                break;
            }
            o += c;
            l += __popc(live[w]);
        }
    }
    __syncthreads();
    const uint32_t bound = limit[0], below = limit[1], wanted = all_live - below;
    const uint32_t moved = (int64_t)wanted < a.max_moves ? wanted : (uint32_t)a.max_moves;

    // Bits of word w at or past the bound.
    auto past = [&](int w) {
        const int d = (int)bound - w * 32;
        return d <= 0 ? ~0u : d >= 32 ? 0u : ~0u << d;
    };
    // The live blocks before block b.
    auto live_rank = [&](uint32_t b) {
        const int w = b >> 5, u = w / unit;
        uint32_t r = live_before[u];
        for (int v = u * unit; v < w; ++v) r += __popc(live[v]);
        return r + __popc(live[w] & ~(~0u << (b & 31)));
    };
    // The r-th free block (r below `wanted`: it lies below the bound).
    auto free_block = [&](uint32_t r) {
        int lo = 0, hi = (words + unit - 1) / unit;  // the last unit with at most r free blocks before it
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (open_before[mid] - live_before[mid] <= r) lo = mid; else hi = mid;
        }
        r -= open_before[lo] - live_before[lo];
        int w = lo * unit;
        for (;; ++w) {
            const uint32_t c = __popc(open[w] & ~live[w]);
            if (r < c) break;
            r -= c;
        }
        return w * 32 + nth_bit(open[w] & ~live[w], r);
    };

    const int64_t at = (int64_t)blockIdx.x * kPoolBlock + tid, step = (int64_t)gridDim.x * kPoolBlock;
    const uint32_t part = blockIdx.x * kPoolWaves + wave, parts = gridDim.x * kPoolWaves;
    const uint32_t all_free = all_open - all_live;
    if (at == 0) a.counts[0] = (int32_t)all_free, a.counts[1] = (int32_t)wanted;
    for (int64_t r = moved + at; r < a.max_moves; r += step) reinterpret_cast<int2*>(a.moves)[r] = int2{-1, -1};
    for (int64_t r = all_free + at; r < a.n_free; r += step) a.free_blocks[r] = -1;
    // Moves: sources by their rank past the bound, destinations by theirs below.
    {
        const int units = (words + unit - 1) / unit, per = (units + parts - 1) / parts;
        const int u0 = part * per, u1 = u0 + per < units ? u0 + per : units;
        if (u0 < u1) {
            uint32_t o = open_before[u0], l = live_before[u0];
            const int e = u1 * unit < words ? u1 * unit : words;
            for (int w = u0 * unit; w < e; w += 2) {
                const bool two = w + 1 < e;
                const uint64_t ob = (uint64_t)(two ? open[w + 1] : 0) << 32 | open[w];
                const uint64_t lb = (uint64_t)(two ? live[w + 1] : 0) << 32 | live[w];
                const uint64_t pb = (uint64_t)(two ? past(w + 1) : 0) << 32 | past(w);
                const uint32_t lr = l + mbcnt64(lb), fr = o + mbcnt64(ob) - lr;  // live and free ones before this lane's
                const bool is_open = ob >> lane & 1, is_live = lb >> lane & 1, is_past = pb >> lane & 1;
                const int id = w * 32 + lane;
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
    for (int64_t i = part; i < a.rows; i += parts) {
        const Lengths n = lengths(a.ctx_lens[i], a.block_size, a.cols);
        for (int j = lane; j < a.cols; j += kWave) {
            int id = -1;
            if (j < n.need) id = a.table[i * a.ld_table + j];
            if ((uint32_t)id >= (uint32_t)a.pool) id = -1;
            if (id >= 0 && (uint32_t)id >= bound && get_bit(live, id)) {
                const uint32_t r = live_rank(id) - below;
                if (r < moved) id = free_block(r);
            }
            a.out_table[i * a.ld_out + j] = id;
        }
    }
}

int launch_compact_blocks(const CompactArgs& a, hipStream_t s) {
    const int64_t work = a.rows * (int64_t)a.cols + a.n_free + 2 * a.max_moves;
    const int64_t grid = work / 16384 < 1 ? 1 : work / 16384 < 64 ? work / 16384 : 64;
    const size_t lds = (size_t)((a.pool + 31) / 32) * 8;
    hipLaunchKernelGGL(compact_blocks_kernel, dim3((unsigned)grid), dim3(kPoolBlock), lds, s, a);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

// Block copies.  A unit is up to kCopySlice bytes of one pair's block in one
// cache; workgroups take units in turn.
constexpr int kCopyBlock = 256;
constexpr int kCopySlice = 16384;

template <typename T>
__device__ __forceinline__ void copy_words(char* data, int64_t src, int64_t dst, int64_t ld, int64_t row_words, int64_t first,
                                           int64_t last) {
    // Words [first, last) of the block, row_words of them a row of ld bytes.
    constexpr int kAhead = 4;
    for (int64_t i0 = first + threadIdx.x; i0 < last; i0 += kCopyBlock * kAhead) {
        T v[kAhead] = {};
        int64_t at[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t i = i0 + u * kCopyBlock;
            at[u] = last <= row_words ? i * (int64_t)sizeof(T)  // one row: no division
                                      : i / row_words * ld + i % row_words * (int64_t)sizeof(T);
            if (i < last) v[u] = *reinterpret_cast<const T*>(data + src * ld + at[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i0 + u * kCopyBlock < last) *reinterpret_cast<T*>(data + dst * ld + at[u]) = v[u];
    }
}

__global__ __launch_bounds__(kCopyBlock) void copy_blocks_kernel(CopyArgs a) {
    const int64_t units = a.n_pairs * a.slices;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t s = u / a.n_pairs, pair = u - s * a.n_pairs;
        const int2 p = reinterpret_cast<const int2*>(a.pairs)[pair];
        if (p.x < 0 || p.y < 0 || p.x == p.y) continue;
        int c = 0;
        while (c + 1 < a.n_caches && s >= a.cache[c + 1].slice0) ++c;
        const CopyCache& k = a.cache[c];
        const int64_t src = p.x * a.stride_rows, dst = p.y * a.stride_rows;
        if (src > k.rows - a.block_size || dst > k.rows - a.block_size) continue;
        const int64_t all = k.words, per = kCopySlice / k.word;
        const int64_t first = (s - k.slice0) * per, last = first + per < all ? first + per : all;
        if (k.word == 16) copy_words<uint4>(k.data, src, dst, k.ld, k.row_words, first, last);
        else if (k.word == 4) copy_words<uint32_t>(k.data, src, dst, k.ld, k.row_words, first, last);
        else if (k.word == 2) copy_words<uint16_t>(k.data, src, dst, k.ld, k.row_words, first, last);
        else copy_words<uint8_t>(k.data, src, dst, k.ld, k.row_words, first, last);
    }
}

int launch_copy_blocks(CopyArgs& a, hipStream_t s) {
    a.slices = 0;
    for (int c = 0; c < a.n_caches; ++c) {
        a.cache[c].slice0 = a.slices;
        a.slices += (a.cache[c].words * a.cache[c].word + kCopySlice - 1) / kCopySlice;
    }
    const int64_t units = a.n_pairs * a.slices;
    const int64_t grid = units < 4096 ? units : 4096;
    hipLaunchKernelGGL(copy_blocks_kernel, dim3((unsigned)grid), dim3(kCopyBlock), 0, s, a);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

}  // namespace rts
