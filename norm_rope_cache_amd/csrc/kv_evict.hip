// Eviction: every (sequence, KV head) keeps the `budget` cells that come first
// in the order (protected, weight falling, index rising), and the kept cells
// past the new end move into the evicted ones' places before it, both in rising
// order. That is the fewest cells that can move, and no cell is both a source
// and a target, so every move is independent of the others.
//
// Selection, one workgroup per (sequence, head): the keys (weights mapped to
// unsigned integers of the same order, protected cells above them all, absent
// ones below) in registers, the budget-th largest found by up to three passes
// over their digits (11, 11 and 10 bits) with a histogram in LDS; then the list
// of holes and the list of the cells that fill them, numbered by ballots in index
// order. It is bound by its passes' instructions and latency on one CU, so long
// lists are split over 16 workgroups, one launch per digit (65536 cells of 16
// heads 57 -> 31 us), and short lists with few moves finish in the same launch
// (4160 cells of 256 heads 21 -> 12.6 us).
// Application, one workgroup per 256 places of a list: the new weights and
// positions, and the 256-byte cells that move, 16 bytes a lane: bound by memory
// (16 heads, half of 65536 cells kept, 77 MB in 15.8 us).
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

__device__ __forceinline__ uint32_t bits_below(uint64_t m, uint32_t lane) {
    return (uint32_t)__popcll(m & (((uint64_t)1 << lane) - 1));
}

// The workspace: [B H, blocks + 1] how many holes lie before each block of 256
// places, and in all; [B H, max_moves] holes; the same many sources, the last
// one in the last place (so that a part of a list can number its own by the
// kept cells before them). Then, where lists are split, [B H, 4, 4] what is
// known after each digit, [B H, 16] the cells of a part above the border, and
// the parts' histograms of two digits, [2, B H, 16, 2048].
constexpr int kPlaces = 256, kParts = 16;
struct Moves {
    int32_t* starts;
    int32_t* holes;
    int32_t* sources;
};
__host__ __device__ __forceinline__ int64_t padded4(int64_t n) { return (n + 3) / 4 * 4; }
__device__ __forceinline__ Moves moves_of(const KvEvictArgs& a, int32_t bh) {
    const int64_t lists = (int64_t)a.B * a.H, per = a.blocks + 1;
    int32_t* holes = a.moves + padded4(lists * per);
    return Moves{a.moves + bh * per, holes + (int64_t)bh * a.max_moves, holes + (lists + bh) * a.max_moves};
}
__device__ __forceinline__ int32_t cells_of(const KvEvictArgs& a, int32_t b) {
    int64_t n = a.lens[b];
    const int64_t cap = (int64_t)a.kv.table_width * a.kv.block_size;
    n = n > a.width ? a.width : n;
    n = n > cap ? cap : n;
    return n < 0 ? 0 : (int32_t)n;
}

// Lanes of one digit count with one addition.
__device__ __forceinline__ void count_digit(uint32_t* hist, uint32_t digit, uint32_t lane) {
    const uint64_t active = __ballot(1);
    const uint32_t lead = __builtin_amdgcn_readfirstlane(digit);
    if (__ballot(digit == lead) == active) {
        if (bits_below(active, lane) == 0) atomicAdd(&hist[digit], (uint32_t)__popcll(active));
    } else {
        atomicAdd(&hist[digit], 1u);
    }
}

constexpr int kWholeMoves = 1024;

// The cells named by two lists in LDS: 16 lanes to a cell, GROUPS cells at a time, four times on the way.
template <int GROUPS>
__device__ __forceinline__ void move_cells(const PagedCache& kv, int32_t b, int32_t h, const int32_t* to_list,
                                           const int32_t* from_list, int32_t count, uint32_t tid) {
    const int32_t* table = kv.tables + (int64_t)b * kv.table_stride;
    uint16_t* head = kv.cache + (int64_t)h * kv.head_stride + 8 * (tid & 15u);
    constexpr int kAtOnce = 4;
    for (int32_t m0 = 0; m0 < count; m0 += GROUPS * kAtOnce) {
        int64_t from[kAtOnce], to[kAtOnce];
        U32x4 cell[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int32_t m = m0 + GROUPS * i + (int32_t)(tid >> 4);
            from[i] = to[i] = -1;
            if (m < count) {
                to[i] = key_offset(kv, table, (uint32_t)to_list[m]);
                from[i] = key_offset(kv, table, (uint32_t)from_list[m]);
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if ((from[i] | to[i]) >= 0) cell[i] = load16(head + from[i]);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if ((from[i] | to[i]) >= 0) store16(head + to[i], cell[i]);
    }
}

// A thread holds its cells' keys, at most SLOTS (<= 64) of them, 64 cells to a
// wave and slot.
// WHOLE (short lists with few moves): the workgroup also does kernel 2's work,
// from the values it holds and lists in LDS; no second launch.
template <int SLOTS, bool WHOLE>
__global__ __launch_bounds__(kThreads) void evict_select_kernel(KvEvictArgs a) {
    static_assert(!WHOLE || SLOTS == 8, "the values of 8 slots at most are held");
    __shared__ int32_t hole[WHOLE ? kWholeMoves : 1], source[WHOLE ? kWholeMoves : 1];
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t wave_sum[kWaves], wave_sum2[kWaves];
    __shared__ uint32_t picked[3];  // the digit, how many are wanted among its cells, how many those are
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    const int32_t n = cells_of(a, b);
    const Moves mv = moves_of(a, bh);
    const float* __restrict__ weights = a.weights + (int64_t)b * a.w_bs + (int64_t)h * a.w_hs;
    const int32_t* __restrict__ positions = a.positions + (int64_t)b * a.p_bs + (int64_t)h * a.p_hs;
    float* __restrict__ new_w = a.new_weights + (int64_t)bh * a.budget;
    int32_t* __restrict__ new_p = a.new_positions + (int64_t)bh * a.budget;
    if (WHOLE && tid == 0 && h == 0) a.new_lens[b] = n < a.budget ? n : a.budget;
    if (n <= a.budget) {
        if constexpr (WHOLE) {
            for (int32_t j = (int32_t)tid; j < a.budget; j += kThreads) {
                new_w[j] = j < n ? weights[j] : 0.0f;
                new_p[j] = j < n ? positions[j] : -1;
            }
        }
        return;
    }
    const int32_t kept = a.budget;

    // The wave's cells: slots of 64 from wave * per_wave * 64 on.
    const int32_t per_wave = (n + kThreads - 1) / kThreads;
    const int32_t base = (int32_t)wave * per_wave * 64 + (int32_t)lane;
    const int64_t horizon = (int64_t)a.ends[b] - a.recent;
    auto key_of = [&](int32_t at, int32_t p, float w) -> uint32_t {
        return at >= n ? 0u : p < a.sinks || p >= horizon ? 0xFFFFFFFFu : ordered(w);
    };
    uint32_t held[SLOTS];
    auto load8 = [&](int i0, int32_t (&p)[8], float (&w)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int32_t at = base + (i0 + i) * 64, in = at < n ? at : n - 1;
            p[i] = positions[in];
            w[i] = weights[in];
        }
    };
    int32_t p[WHOLE ? 8 : 1];
    float w[WHOLE ? 8 : 1];
    if constexpr (WHOLE) {
        load8(0, p, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) held[i] = i < per_wave ? key_of(base + i * 64, p[i], w[i]) : 0u;
    } else {
        // eight slots' loads on the way together (a position decides only what its weight counts for)
#pragma unroll
        for (int i0 = 0; i0 < SLOTS; i0 += 8) {
            int32_t p8[8];
            float w8[8];
            if (i0 < per_wave) load8(i0, p8, w8);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                held[i0 + i] = i0 + i < per_wave ? key_of(base + (i0 + i) * 64, p8[i], w8[i]) : 0u;
        }
    }
    // what the waves before this one add up to, of a sum each wave has left in LDS
    auto before_this = [&](const uint32_t* sums, uint32_t* all) {
        const uint32_t v = sums[lane & 15u];
        const uint32_t first16 = lane < 16 ? v : 0u;
        if (all) *all = wave_total(first16);
        return wave_total(lane < wave ? first16 : 0u);
    };
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if (i < per_wave) f(i, held[i]);
    };

    uint32_t border = 0, want = (uint32_t)kept;  // the digits found so far; how many of the cells with them
    bool all_ties = false;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        hist[tid] = 0u;
        hist[tid + kThreads] = 0u;
        __syncthreads();
        each([&](int, uint32_t key) {
            if (pass > 0 && (key >> (shift + bits)) != border) return;
            count_digit(hist, key >> shift & ((1u << bits) - 1u), lane);
        });
        __syncthreads();
        // from the largest digit down: thread t the digits 2047 - 2t and 2046 - 2t
        const uint32_t hi = hist[kBins - 1 - 2 * tid], lo = hist[kBins - 2 - 2 * tid];
        const uint32_t incl = wave_inclusive(hi + lo);
        if (lane == 63) wave_sum[wave] = incl;
        __syncthreads();
        const uint32_t before = incl - hi - lo + before_this(wave_sum, nullptr);
        if (before < want && want <= before + hi + lo) {
            const bool first = want <= before + hi;
            picked[0] = kBins - 1 - 2 * tid - (first ? 0u : 1u);
            picked[1] = want - before - (first ? 0u : hi);
            picked[2] = first ? hi : lo;
        }
        __syncthreads();
        border = border << bits | picked[0];
        want = picked[1];
        all_ties = picked[2] == want;
        if (all_ties) {  // every cell with these digits is kept: the others do not matter
            border <<= shift;
            break;
        }
    }
    // Kept: keys above `border`, and the first `want` cells that equal it (a cell past n has key 0, which no
    // border reaches); with all_ties the keys from `border` on.
    __syncthreads();
    uint32_t tie0 = 0;  // equal cells of the waves before
    if (!all_ties) {
        uint32_t ties = 0;
        each([&](int, uint32_t key) { ties += (uint32_t)__popcll(__ballot(key == border)); });
        if (lane == 0) wave_sum[wave] = ties;
        __syncthreads();
        tie0 = before_this(wave_sum, nullptr);
        __syncthreads();
    }
    // f(slot, is a hole, is a source): of each of the lane's cells, the wave together
    auto walk = [&](auto f) {
        uint32_t seen = tie0;
        each([&](int i, uint32_t key) {
            const int32_t at = base + i * 64;
            bool keep = key >= border;
            if (!all_ties) {
                const uint64_t tied = __ballot(key == border);
                keep = key > border || (key == border && seen + bits_below(tied, lane) < want);
                seen += (uint32_t)__popcll(tied);
            }
            f(i, !keep && at < kept, keep && at >= kept);
        });
    };
    uint32_t holes = 0, sources = 0;
    walk([&](int, bool hole, bool source) {
        holes += hole;
        sources += source;
    });
    holes = wave_total(holes);
    sources = wave_total(sources);
    if (lane == 0) {
        wave_sum[wave] = holes;
        wave_sum2[wave] = sources;
    }
    __syncthreads();
    uint32_t count = 0;
    uint32_t hole0 = before_this(wave_sum, &count), source0 = before_this(wave_sum2, nullptr);
    if constexpr (!WHOLE) {
        if (tid == 0) mv.starts[a.blocks] = (int32_t)count;
        int32_t* last_sources = mv.sources + a.max_moves - (int32_t)count;
        walk([&](int i, bool is_hole, bool is_source) {
            const int32_t at = base + i * 64, group = (int32_t)wave * per_wave + i;
            // 64 cells a slot: every fourth begins a block of places
            if ((group & 3) == 0 && group * 64 < kept && lane == 0) mv.starts[group >> 2] = (int32_t)hole0;
            const uint64_t hm = __ballot(is_hole), sm = __ballot(is_source);
            if (is_hole) mv.holes[hole0 + bits_below(hm, lane)] = at;
            if (is_source) last_sources[source0 + bits_below(sm, lane)] = at;
            hole0 += (uint32_t)__popcll(hm);
            source0 += (uint32_t)__popcll(sm);
        });
    } else {
        int32_t rank[8];  // of the lane's sources, -1: none
        walk([&](int i, bool is_hole, bool is_source) {
            const int32_t at = base + i * 64;
            const uint64_t hm = __ballot(is_hole), sm = __ballot(is_source);
            if (is_hole) hole[hole0 + bits_below(hm, lane)] = at;
            rank[i] = is_source ? (int32_t)(source0 + bits_below(sm, lane)) : -1;
            if (is_source) source[rank[i]] = at;
            hole0 += (uint32_t)__popcll(hm);
            source0 += (uint32_t)__popcll(sm);
            if (!is_hole && at < kept) {
                new_w[at] = w[i];
                new_p[at] = p[i];
            }
        });
        __syncthreads();
        each([&](int i, uint32_t) {
            if (rank[i] >= 0) {
                const int32_t to = hole[rank[i]];
                new_w[to] = w[i];
                new_p[to] = p[i];
            }
        });
        move_cells<kThreads / 16>(a.kv, b, h, hole, source, (int32_t)count, tid);
    }
}

// A list split over kParts workgroups, one launch per digit and one for the
// lists of moves: launch PASS finds digit PASS - 1 from the parts' histograms
// (every workgroup for itself) and counts digit PASS of its own cells. A list
// whose border is known early is done with counting.
struct Split {
    int32_t* state;    // [4][4], after each digit: border, wanted among the equal ones, known
    int32_t* above;    // [kParts]
    uint32_t* counts;  // [2][lists][kParts][kBins], this list's
    int64_t stride;    // between its two halves
};
__device__ __forceinline__ Split split_of(const KvEvictArgs& a, int32_t bh) {
    const int64_t lists = (int64_t)a.B * a.H;
    int32_t* state = a.moves + padded4(lists * (a.blocks + 1)) + padded4(2 * lists * a.max_moves);
    int32_t* above = state + lists * 16;
    int32_t* counts = above + lists * kParts;
    return Split{state + bh * 16, above + bh * kParts,
                 reinterpret_cast<uint32_t*>(counts) + (int64_t)bh * kParts * kBins, lists * kParts * kBins};
}

template <int PASS, int SLOTS>
__global__ __launch_bounds__(kThreads) void evict_split_kernel(KvEvictArgs a) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t wave_sum[kWaves], wave_sum2[kWaves];
    __shared__ uint32_t picked[3];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t part = blockIdx.x, bh = blockIdx.y, b = bh / a.H, h = bh - b * a.H;
    const int32_t n = cells_of(a, b), kept = a.budget;
    if (n <= kept) return;
    const Split split = split_of(a, bh);
    const float* __restrict__ weights = a.weights + (int64_t)b * a.w_bs + (int64_t)h * a.w_hs;
    const int32_t* __restrict__ positions = a.positions + (int64_t)b * a.p_bs + (int64_t)h * a.p_hs;

    // The part's cells: per_wave slots of 64 of each wave, in order.
    const int32_t per_wave = (n + kParts * kThreads - 1) / (kParts * kThreads);
    const int64_t part0 = (int64_t)part * per_wave * kThreads;
    const int64_t base = part0 + (int64_t)wave * per_wave * 64 + lane;
    const int64_t horizon = (int64_t)a.ends[b] - a.recent;
    auto key_of = [&](int64_t at, int32_t p, float w) -> uint32_t {
        return at >= n ? 0u : p < a.sinks || p >= horizon ? 0xFFFFFFFFu : ordered(w);
    };
    // SLOTS: on the way while the digit before is found; 0: more than a thread holds
    uint32_t held[SLOTS ? SLOTS : 1];
    if constexpr (SLOTS > 0) {
        int32_t p[SLOTS];
        float w[SLOTS];
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int64_t at = base + i * 64;
            const int32_t in = at < n ? (int32_t)at : n - 1;
            p[i] = positions[in];
            w[i] = weights[in];
        }
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) held[i] = i < per_wave ? key_of(base + i * 64, p[i], w[i]) : 0u;
    }
    auto each = [&](auto f) {
        if constexpr (SLOTS > 0) {
#pragma unroll
            for (int i = 0; i < SLOTS; ++i)
                if (i < per_wave) f(i, held[i]);
        } else {
            for (int32_t i = 0; i < per_wave; ++i) {
                const int64_t at = base + (int64_t)i * 64;
                const int32_t in = at < n ? (int32_t)at : n - 1;
                f(i, key_of(at, positions[in], weights[in]));
            }
        }
    };
    auto total_of = [&](uint32_t v) {  // over the workgroup
        v = wave_total(v);
        __syncthreads();
        if (lane == 0) wave_sum2[wave] = v;
        __syncthreads();
        return wave_total(lane < 16 ? wave_sum2[lane & 15u] : 0u);
    };

    uint32_t border = 0, want = (uint32_t)kept;
    bool known = false;  // `border` whole, and all cells from it on are kept
    bool was_known = false;
    uint32_t digit = 0;  // the one found here
    if constexpr (PASS > 0) {
        if constexpr (PASS > 1) {
            const int32_t* st = split.state + 4 * (PASS - 1);
            border = (uint32_t)st[0];
            want = (uint32_t)st[1];
            was_known = known = st[2] != 0;
        }
        if (!known) {
            constexpr int shift = PASS == 1 ? 21 : PASS == 2 ? 10 : 0, bits = PASS == 3 ? 10 : 11;
            const uint32_t* counts = split.counts + ((PASS - 1) & 1) * split.stride;
            // from the largest digit down: thread t the digits 2047 - 2t and 2046 - 2t
            const uint32_t d = kBins - 2 - 2 * tid;
            uint32_t hi = 0, lo = 0, own_hi = 0, own_lo = 0;
#pragma unroll
            for (int c = 0; c < kParts; ++c) {
                const uint2 v = *reinterpret_cast<const uint2*>(counts + c * kBins + d);
                lo += v.x;
                hi += v.y;
                if (c == part) {
                    own_lo = v.x;
                    own_hi = v.y;
                }
            }
            const uint32_t incl = wave_inclusive(hi + lo);
            if (lane == 63) wave_sum[wave] = incl;
            __syncthreads();
            const uint32_t before = incl - hi - lo + wave_total(lane < wave ? wave_sum[lane & 15u] : 0u);
            if (before < want && want <= before + hi + lo) {
                const bool first = want <= before + hi;
                picked[0] = d + (first ? 1u : 0u);
                picked[1] = want - before - (first ? 0u : hi);
                picked[2] = first ? hi : lo;
            }
            __syncthreads();
            digit = picked[0];
            border = border << bits | digit;
            want = picked[1];
            known = picked[2] == want;
            if constexpr (PASS < 3) {
                const uint32_t from = known ? digit : digit + 1;
                const uint32_t mine = total_of((d >= from ? own_lo : 0u) + (d + 1 >= from ? own_hi : 0u));
                if (tid == 0) split.above[part] = (PASS == 1 ? 0 : split.above[part]) + (int32_t)mine;
            }
            if (known) border <<= shift;
        }
        if constexpr (PASS < 3) {
            if (part == 0 && tid == 0) {
                int32_t* st = split.state + 4 * PASS;
                st[0] = (int32_t)border;
                st[1] = (int32_t)want;
                st[2] = known;
            }
            if (known) return;
        }
    }
    if constexpr (PASS < 3) {
        constexpr int shift = PASS == 0 ? 21 : PASS == 1 ? 10 : 0, bits = PASS == 2 ? 10 : 11;
        hist[tid] = 0u;
        hist[tid + kThreads] = 0u;
        __syncthreads();
        each([&](int, uint32_t key) {
            if (PASS == 0 || (key >> (shift + bits)) == border) count_digit(hist, key >> shift & ((1u << bits) - 1u), lane);
        });
        __syncthreads();
        uint32_t* mine = split.counts + (PASS & 1) * split.stride + part * kBins;
        *reinterpret_cast<uint2*>(mine + 2 * tid) = uint2{hist[2 * tid], hist[2 * tid + 1]};
        return;
    }

    // The kept and the equal cells of the parts before this one: wave c counts part c.
    const Moves mv = moves_of(a, bh);
    uint32_t above = 0, equal = 0;
    if ((int32_t)wave < part) {
        if (!was_known) {
            const uint32_t* counts = split.counts + wave * kBins;  // the third digit's, in the first half
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t d = i * 64 + lane, v = counts[d];
                if (d > digit) above += v;
                if (d == digit) equal += v;
            }
        }
        above = wave_total(above) + (uint32_t)split.above[wave];
        equal = wave_total(equal);
    }
    __syncthreads();
    if (lane == 0) {
        wave_sum[wave] = above;
        wave_sum2[wave] = equal;
    }
    __syncthreads();
    above = wave_total(lane < 16 ? wave_sum[lane & 15u] : 0u);
    equal = wave_total(lane < 16 ? wave_sum2[lane & 15u] : 0u);
    // Equal cells before the wave, then kept ones.
    uint32_t ties = 0;
    each([&](int, uint32_t key) { ties += (uint32_t)__popcll(__ballot(key == border)); });
    __syncthreads();
    if (lane == 0) wave_sum[wave] = ties;
    __syncthreads();
    const uint32_t tie0 = equal + wave_total(lane < wave ? wave_sum[lane & 15u] : 0u);
    auto walk = [&](auto f) {
        uint32_t seen = tie0;
        each([&](int i, uint32_t key) {
            const uint64_t tied = __ballot(key == border);
            f(i, key > border || (key == border && (known || seen + bits_below(tied, lane) < want)));
            seen += (uint32_t)__popcll(tied);
        });
    };
    uint32_t stay = 0;
    walk([&](int, bool keep) { stay += (uint32_t)__popcll(__ballot(keep)); });
    __syncthreads();
    if (lane == 0) wave_sum2[wave] = stay;
    __syncthreads();
    // kept cells before each slot
    int32_t rank = (int32_t)(above + (known ? equal : equal < want ? equal : want) +
                             wave_total(lane < wave ? wave_sum2[lane & 15u] : 0u));
    walk([&](int i, bool keep) {
        const int64_t at0 = part0 + ((int64_t)wave * per_wave + i) * 64, at = at0 + lane;
        const uint64_t m = __ballot(keep);
        // before the new end every cell is kept or a hole
        if (at0 <= kept) {
            if ((at0 & (kPlaces - 1)) == 0 && at0 < kept && lane == 0) mv.starts[at0 >> 8] = (int32_t)at0 - rank;
            if (at == kept) mv.starts[a.blocks] = (int32_t)at - rank - (int32_t)bits_below(m, lane);
        }
        const int32_t r = rank + (int32_t)bits_below(m, lane);
        if (at < kept && !keep) mv.holes[at - r] = (int32_t)at;
        if (at >= kept && keep) mv.sources[a.max_moves - kept + r] = (int32_t)at;
        rank += (int32_t)__popcll(m);
    });
}

// One workgroup: 256 places of a list.
__global__ __launch_bounds__(kPlaces) void evict_apply_kernel(KvEvictArgs a) {
    __shared__ int32_t origin[kPlaces], hole[kPlaces], from_cell[kPlaces];
    const int32_t tid = (int32_t)threadIdx.x, j0 = (int32_t)blockIdx.x * kPlaces, j = j0 + tid;
    const int32_t bh = blockIdx.y, b = bh / a.H, h = bh - b * a.H;
    const int32_t n = cells_of(a, b), kept = n < a.budget ? n : a.budget;
    const float* weights = a.weights + (int64_t)b * a.w_bs + (int64_t)h * a.w_hs;
    const int32_t* positions = a.positions + (int64_t)b * a.p_bs + (int64_t)h * a.p_hs;
    float weight = 0.0f;
    int32_t position = -1;
    if (j < kept) {  // on the way before it is known which places are holes
        weight = weights[j];
        position = positions[j];
    }
    int32_t first = 0, moved = 0;  // of the holes among these places
    origin[tid] = j;
    if (n > a.budget) {
        const Moves mv = moves_of(a, bh);
        first = mv.starts[blockIdx.x];
        moved = mv.starts[blockIdx.x + 1] - first;
        __syncthreads();
        if (tid < moved) {
            const int32_t to = mv.holes[first + tid];
            hole[tid] = to;
            from_cell[tid] = mv.sources[a.max_moves - mv.starts[a.blocks] + first + tid];
            origin[to - j0] = from_cell[tid];
        }
        __syncthreads();
    }
    if (j < a.budget) {
        const int64_t at = (int64_t)bh * a.budget + j;
        const int32_t from = origin[tid];
        if (from != j) {
            weight = weights[from];
            position = positions[from];
        }
        a.new_weights[at] = weight;
        a.new_positions[at] = position;
    }
    if (bh - b * a.H == 0 && j == 0) a.new_lens[b] = kept;
    move_cells<kPlaces / 16>(a.kv, b, h, hole, from_cell, moved, threadIdx.x);
}

}  // namespace

namespace {
// Up to 8192 cells with up to 1024 moves (256 KiB a list; half of that where there are more lists than CUs) take one
// launch: a call on 256 lists of 4160 cells, 64 of them gone, 15 us against 21 in two launches; of 2048 cells, half of
// them, 20.8 against 25.3; 64 lists of 1548 cells, half, 16.7 against 22.2. At 2048 moves 512 lists of 4096 cells took
// 87 against 73.
bool in_one(int64_t lists, int64_t width, int64_t max_moves) {
    return max_moves <= (lists <= 256 ? kWholeMoves : kWholeMoves / 2) && width <= 8 * kThreads;
}
// A list takes one launch of one workgroup, or four of 16 (its cells read again in each): past what a workgroup
// holds, always (8 lists of 131072 cells 60 us in all, 358 when one workgroup reads again); past half of that where few
// lists would leave most CUs idle (65536 cells: 16 lists 57 against 87 us, 32 lists 102 against 113, 64 lists 202 against
// 179; 20000 cells: 16 lists 44 against 36).
bool in_parts(int64_t lists, int64_t width) {
    return width > 64 * kThreads || (width > 32 * kThreads && lists <= 32);
}
}  // namespace

int64_t kv_evict_workspace(int64_t lists, int64_t width, int64_t max_moves, int64_t blocks) {
    if (max_moves == 0 || in_one(lists, width, max_moves)) return 0;
    int64_t words = padded4(lists * (blocks + 1)) + padded4(2 * lists * max_moves);
    if (in_parts(lists, width)) words += lists * (16 + kParts + 2 * kParts * kBins);
    return words * 4;
}

int32_t kv_evict_blocks(int64_t budget) { return (int32_t)((budget + kPlaces - 1) / kPlaces); }

int launch_kv_evict(const KvEvictArgs& a, hipStream_t stream) {
    const uint32_t lists = (uint32_t)a.B * a.H;
    if (a.max_moves > 0 && in_one(lists, a.width, a.max_moves)) {
        hipLaunchKernelGGL((evict_select_kernel<8, true>), dim3(lists), dim3(kThreads), 0, stream, a);
        return hipGetLastError() == hipSuccess ? 0 : -1;
    }
    if (a.max_moves > 0 && in_parts(lists, a.width)) {
        const bool hold = a.width <= (int64_t)8 * kParts * kThreads;
        const dim3 grid(kParts, lists);
        auto go = [&](auto held, auto again) { hipLaunchKernelGGL(hold ? held : again, grid, dim3(kThreads), 0, stream, a); };
        go(evict_split_kernel<0, 8>, evict_split_kernel<0, 0>);
        go(evict_split_kernel<1, 8>, evict_split_kernel<1, 0>);
        go(evict_split_kernel<2, 8>, evict_split_kernel<2, 0>);
        go(evict_split_kernel<3, 8>, evict_split_kernel<3, 0>);
    } else if (a.max_moves > 0) {
        // what a thread can hold, by the longest sequence there may be
        auto kernel = a.width <= 8 * kThreads    ? evict_select_kernel<8, false>
                      : a.width <= 16 * kThreads ? evict_select_kernel<16, false>
                      : a.width <= 32 * kThreads ? evict_select_kernel<32, false>
                                                 : evict_select_kernel<64, false>;
        hipLaunchKernelGGL(kernel, dim3(lists), dim3(kThreads), 0, stream, a);
    }
    hipLaunchKernelGGL(evict_apply_kernel, dim3((uint32_t)a.blocks, lists), dim3(kPlaces), 0, stream, a);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
