// Eviction: every (sequence, KV head) keeps the `budget` cells that come first
// in the order (protected, weight falling, index rising), and the kept cells
// past the new end move into the evicted ones' places before it, both in rising
// order. That is the fewest cells that can move, and no cell is both a source
// and a target, so every move is independent of the others.
//
// Kernel 1, one workgroup per (sequence, head): the keys (weights mapped to
// unsigned integers of the same order, protected cells above them all, absent
// ones below) in registers, the budget-th largest found by three passes over
// their digits (11, 11 and 10 bits) with a histogram in LDS, ties and moves
// numbered by ballots in index order. Kernel 2 moves the 256-byte cells, 16
// bytes a lane. Kernel 1 is bound by its passes' latency, kernel 2 by memory.
#include "cache_ops.h"
#include "paged.h"

namespace nrc {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64, kBins = 2048;

// Unsigned in the weights' order (a NaN as the least weight, -0 as 0).
__device__ __forceinline__ uint32_t ordered(float w) {
    if (__builtin_isnan(w)) w = -__builtin_inff();
    uint32_t u = __float_as_uint(w);
    if (u == 0x80000000u) u = 0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t wave_inclusive(uint32_t v, uint32_t lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_ds_bpermute((int)((lane - d) << 2), (int)v);
        if (lane >= (uint32_t)d) v += o;
    }
    return v;
}

__device__ __forceinline__ uint32_t bits_below(uint64_t m, uint32_t lane) {
    return (uint32_t)__popcll(m & (((uint64_t)1 << lane) - 1));
}

// SLOTS > 0: a thread holds its cells' keys, at most SLOTS 64-cell slots a
// wave; 0: they are worked out again in every pass.
template <int SLOTS>
__global__ __launch_bounds__(kThreads) void evict_select_kernel(KvEvictArgs a) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t wave_sum[kWaves], wave_sum2[kWaves];
    __shared__ uint32_t picked[2];  // the digit, and how many are wanted among its cells
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    int64_t n64 = a.lens[b];
    if (n64 < 0) n64 = 0;
    if (n64 > a.width) n64 = a.width;
    const int64_t cap = (int64_t)a.kv.table_width * a.kv.block_size;
    if (n64 > cap) n64 = cap;
    const int32_t n = (int32_t)n64;
    const int32_t kept = n < a.budget ? n : a.budget;
    const float* weights = a.weights + (int64_t)b * a.w_bs + (int64_t)h * a.w_hs;
    const int32_t* positions = a.positions + (int64_t)b * a.p_bs + (int64_t)h * a.p_hs;
    float* new_w = a.new_weights + (int64_t)bh * a.budget;
    int32_t* new_p = a.new_positions + (int64_t)bh * a.budget;
    if (h == 0 && tid == 0) a.new_lens[b] = kept;
    for (int32_t i = kept + (int32_t)tid; i < a.budget; i += kThreads) {
        new_w[i] = 0.0f;
        new_p[i] = -1;
    }
    const int32_t lists = (gridDim.x + 3) / 4 * 4;
    if (n <= a.budget) {
        for (int32_t i = (int32_t)tid; i < n; i += kThreads) {
            new_w[i] = weights[i];
            new_p[i] = positions[i];
        }
        if (tid == 0 && a.max_moves > 0) a.moves[bh] = 0;
        return;
    }

    // The wave's cells: slots of 64 from wave * per_wave * 64 on.
    const int32_t per_wave = (n + kThreads - 1) / kThreads;
    const int32_t base = (int32_t)wave * per_wave * 64 + (int32_t)lane;
    const int64_t horizon = (int64_t)a.ends[b] - a.recent;
    auto work_out = [&](int32_t i) -> uint32_t {
        const int32_t at = base + i * 64;
        if (at >= n) return 0u;
        const int32_t p = positions[at];
        return p < a.sinks || p >= horizon ? 0xFFFFFFFFu : ordered(weights[at]);
    };
    uint32_t held[SLOTS ? SLOTS : 1];
    if constexpr (SLOTS > 0) {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) held[i] = i < per_wave ? work_out(i) : 0u;
    }
    auto each = [&](auto f) {
        if constexpr (SLOTS > 0) {
#pragma unroll
            for (int i = 0; i < SLOTS; ++i)
                if (i < per_wave) f(i, held[i]);
        } else {
            for (int32_t i = 0; i < per_wave; ++i) f(i, work_out(i));
        }
    };

    uint32_t border = 0, want = (uint32_t)kept;  // the digits found so far; how many of the cells with them
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        hist[tid] = 0u;
        hist[tid + kThreads] = 0u;
        __syncthreads();
        each([&](int, uint32_t key) {
            if (pass > 0 && (key >> (shift + bits)) != border) return;
            const uint32_t digit = key >> shift & ((1u << bits) - 1u);
            // cells of one digit count with one addition
            const uint64_t active = __ballot(1);
            const uint32_t lead = __builtin_amdgcn_readfirstlane(digit);
            if (__ballot(digit == lead) == active) {
                if (bits_below(active, lane) == 0) atomicAdd(&hist[digit], (uint32_t)__popcll(active));
            } else {
                atomicAdd(&hist[digit], 1u);
            }
        });
        __syncthreads();
        // from the largest digit down: thread t the digits 2047 - 2t and 2046 - 2t
        const uint32_t hi = hist[kBins - 1 - 2 * tid], lo = hist[kBins - 2 - 2 * tid];
        const uint32_t incl = wave_inclusive(hi + lo, lane);
        if (lane == 63) wave_sum[wave] = incl;
        __syncthreads();
        uint32_t before = incl - hi - lo;
        for (uint32_t w = 0; w < wave; ++w) before += wave_sum[w];
        if (before < want && want <= before + hi + lo) {
            const bool first = want <= before + hi;
            picked[0] = kBins - 1 - 2 * tid - (first ? 0u : 1u);
            picked[1] = want - before - (first ? 0u : hi);
        }
        __syncthreads();
        border = border << bits | picked[0];
        want = picked[1];
        __syncthreads();
    }
    // Kept: keys above `border`, and the first `want` cells that equal it.

    uint32_t ties = 0;
    each([&](int, uint32_t key) { ties += (uint32_t)__popcll(__ballot(key == border)); });
    if (lane == 0) wave_sum[wave] = ties;
    __syncthreads();
    uint32_t tie0 = 0;
    for (uint32_t w = 0; w < wave; ++w) tie0 += wave_sum[w];
    __syncthreads();

    // (the ballots take every lane of the wave: cells past n have key 0, which
    // no border reaches)
    auto walk = [&](auto f) {
        uint32_t seen = tie0;
        each([&](int i, uint32_t key) {
            const int32_t at = base + i * 64;
            const uint64_t tied = __ballot(key == border);
            const bool keep = key > border || (key == border && seen + bits_below(tied, lane) < want);
            seen += (uint32_t)__popcll(tied);
            f(at, keep && at < n, !keep && at < kept, keep && at >= kept && at < n);
        });
    };
    uint32_t holes = 0, sources = 0;
    walk([&](int32_t, bool, bool hole, bool source) {
        holes += (uint32_t)__popcll(__ballot(hole));
        sources += (uint32_t)__popcll(__ballot(source));
    });
    if (lane == 0) {
        wave_sum[wave] = holes;
        wave_sum2[wave] = sources;
    }
    __syncthreads();
    uint32_t hole0 = 0, source0 = 0, count = 0;
    for (uint32_t w = 0; w < (uint32_t)kWaves; ++w) {
        if (w < wave) {
            hole0 += wave_sum[w];
            source0 += wave_sum2[w];
        }
        count += wave_sum[w];
    }
    int32_t* hole_list = a.moves + lists + (int64_t)bh * a.max_moves;
    int32_t* source_list = hole_list + (int64_t)gridDim.x * a.max_moves;
    if (tid == 0) a.moves[bh] = (int32_t)count;
    // the holes' list first: the sources look their targets up in it
    {
        uint32_t next = hole0;
        walk([&](int32_t at, bool keep, bool hole, bool source) {
            const uint64_t m = __ballot(hole);
            if (hole) hole_list[next + bits_below(m, lane)] = at;
            next += (uint32_t)__popcll(m);
            if (keep && !source) {
                new_w[at] = weights[at];
                new_p[at] = positions[at];
            }
        });
    }
    __syncthreads();
    uint32_t next = source0;
    walk([&](int32_t at, bool, bool, bool source) {
        const uint64_t m = __ballot(source);
        if (source) {
            const uint32_t rank = next + bits_below(m, lane);
            const int32_t to = hole_list[rank];
            source_list[rank] = at;
            new_w[to] = weights[at];
            new_p[to] = positions[at];
        }
        next += (uint32_t)__popcll(m);
    });
}

// 16 cells a workgroup and pass, 16 lanes to a cell.
constexpr int kMovesPerBlock = 64;
__global__ __launch_bounds__(256) void evict_move_kernel(PagedCache kv, int32_t H, const int32_t* __restrict__ moves,
                                                         int32_t max_moves) {
    const int32_t bh = blockIdx.y, b = bh / H, h = bh - b * H;
    const int32_t count = moves[bh] < max_moves ? moves[bh] : max_moves;
    const int32_t lists = (gridDim.y + 3) / 4 * 4;
    const int32_t* holes = moves + lists + (int64_t)bh * max_moves;
    const int32_t* sources = holes + (int64_t)gridDim.y * max_moves;
    const int32_t* table = kv.tables + (int64_t)b * kv.table_stride;
    uint16_t* head = kv.cache + (int64_t)h * kv.head_stride + 8 * (threadIdx.x & 15u);
    int64_t from[kMovesPerBlock / 16], to[kMovesPerBlock / 16];
    U32x4 cell[kMovesPerBlock / 16];
#pragma unroll
    for (int i = 0; i < kMovesPerBlock / 16; ++i) {
        const int32_t m = (int32_t)blockIdx.x * kMovesPerBlock + 16 * i + (int32_t)(threadIdx.x >> 4);
        from[i] = to[i] = -1;
        if (m < count) {
            from[i] = key_offset(kv, table, (uint32_t)sources[m]);
            to[i] = key_offset(kv, table, (uint32_t)holes[m]);
        }
    }
#pragma unroll
    for (int i = 0; i < kMovesPerBlock / 16; ++i)
        if ((from[i] | to[i]) >= 0) cell[i] = load16(head + from[i]);
#pragma unroll
    for (int i = 0; i < kMovesPerBlock / 16; ++i)
        if ((from[i] | to[i]) >= 0) store16(head + to[i], cell[i]);
}

}  // namespace

int launch_kv_evict(const KvEvictArgs& a, hipStream_t stream) {
    const uint32_t lists = (uint32_t)a.B * a.H;
    // what a thread can hold, by the longest sequence there may be
    auto kernel = a.width <= 4 * kThreads    ? evict_select_kernel<4>
                  : a.width <= 16 * kThreads ? evict_select_kernel<16>
                  : a.width <= 64 * kThreads ? evict_select_kernel<64>
                                             : evict_select_kernel<0>;
    hipLaunchKernelGGL(kernel, dim3(lists), dim3(kThreads), 0, stream, a);
    if (a.max_moves > 0) {
        const dim3 grid((uint32_t)(a.max_moves + kMovesPerBlock - 1) / kMovesPerBlock, lists);
        hipLaunchKernelGGL(evict_move_kernel, grid, dim3(256), 0, stream, a.kv, a.H, a.moves, a.max_moves);
    }
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
