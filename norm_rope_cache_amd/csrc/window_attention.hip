// Attention of drafted tokens over the paged cache behind a sliding window with
// a few first keys that stay visible, and over a cache held in 4 bits.
//
// The formulas, the running softmax and its roundings are those of
// tree_attention.hip; what differs is which keys there are to look at and what a cell is.
//
// Window: a row at position p sees the keys j <= p with j > p - window or j <
// sinks. A workgroup's rows stand at nearby positions, so the tiles it looks at are
// those of the sinks and those from its first row's window to its last row's own
// key: two runs, walked as one by their numbers. A tile that every row of a wave
// sees whole (most of them) goes without a mask, others get one from each row's
// first key, by shifts alone for a chain.
//
// 4 bits: K's and V's elements are bf16 numbers once opened (a code's value times a
// power of two), so the matrix instructions take them as a bf16 cache's, with
// nothing rounded on the way. The conversion takes two codes an instruction. A cell that
// stands for NaN has NaN in K, so a row that sees it gets NaN scores and outputs; in a
// tile that some rows do not see whole, V's scales are held to 2^125, so that 0
// times a V that a row does not see is 0.
//
// Few rows a KV head (up to 32) are bound by the cache's bytes and, in 4 bits, by
// the instructions that open them; many rows by the vector unit and the matrix cores.
#include <atomic>
#include <type_traits>

#include "../../include/nrc.h"
#include "attention_core.h"
#include "draft_ops.h"
#include "fp4.h"
#include "kernels.h"

namespace nrc {
namespace {

constexpr int32_t kNoWindow = 0x7FFFFFFF;

// The keys that a block of rows looks at: key j if any row may see it lies in [0, sinks) or [lo_min, hi_max]; every row
// sees those in [lo_max, hi_min], and the sinks up to hi_min.
struct Keyspan {
    int32_t lo_min, lo_max, hi_min, hi_max;
};
// Of rows first .. last (of the sequence's; last is cut to them). A tree's rows stand at ctx + the nodes they see - 1.
__device__ __forceinline__ Keyspan keyspan(const WindowArgs& a, const Span& s, int32_t first, int32_t last) {
    if (last >= s.rows) last = s.rows - 1;
    if (a.tq.mask) return Keyspan{s.ctx - a.window, s.ctx - a.window + s.nodes.count, s.ctx - 1, s.ctx + s.nodes.count - 1};
    const int32_t n0 = (int32_t)quotient((uint32_t)first, a.by_group), n1 = (int32_t)quotient((uint32_t)last, a.by_group);
    return Keyspan{s.ctx - a.window + 1 + n0, s.ctx - a.window + 1 + n1, s.ctx + n0, s.ctx + n1};
}

// The keys that a block of rows looks at, one after the other: the sinks (as whole 32s; none where the windows reach back
// to them), then those from `base` (a multiple of 32) to hi_max. They are dealt into tiles of KEYS, n in all.
struct Tiles {
    int32_t sinks, base, n;
    // the key at place p, a multiple of 16 (the 16 from there on lie together)
    __device__ __forceinline__ int32_t key(int32_t p) const { return p < sinks ? p : p - sinks + base; }
    // the place of a key that is not before `base`
    __device__ __forceinline__ int64_t place(int64_t key) const { return key - base + sinks; }
};
template <int KEYS>
__device__ __forceinline__ Tiles tiles_of(const Keyspan& k, int32_t sinks) {
    Tiles t;
    t.base = k.lo_min < 0 ? 0 : k.lo_min & ~31;
    t.sinks = sinks > t.base ? t.base : (sinks + 31) & ~31;
    if (t.sinks >= t.base) t.base = t.sinks = 0;
    t.n = (int32_t)(t.place(k.hi_max) / KEYS) + 1;
    return t;
}
// The numbers of the tiles that every one of the rows sees whole, from .x to .y (but for some of the sinks alone).
template <int KEYS>
__device__ __forceinline__ int2 whole_tiles(const Keyspan& k, const Tiles& t, int32_t sinks) {
    const int64_t from = k.lo_max <= t.base || (t.base == 0 && sinks >= k.lo_max) ? t.sinks : t.place(k.lo_max);
    const int64_t upto = t.place(k.hi_min + 1) / KEYS, first = (from + KEYS - 1) / KEYS;
    return int2{(int32_t)first, (int32_t)(upto < first ? first : upto)};
}

// May any of the rows see one of the 32 keys from key0 on?
__device__ __forceinline__ bool may_be_seen(const Keyspan& k, int32_t sinks, int32_t key0) {
    return key0 <= k.hi_max && (key0 + 31 >= k.lo_min || key0 < sinks);
}

// The bits i of a word of 32 with i < n (any n).
__device__ __forceinline__ uint32_t below(int32_t n) {
    const int32_t k = n < 0 ? 0 : n;
    return k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
}
// Bits i of a word of 32 keys from key0 on with key0 + i < end (a key's number, or one past it: the difference fits 32 bits
// where end is at least -2^31 + 2 and key0 below 2^31 - 2^17).
__device__ __forceinline__ uint32_t below_key(int32_t end, int32_t key0) { return end <= key0 ? 0u : below(end - key0); }

// A lane's row: its node (-1: none) and the first key of its window.
struct Row {
    int32_t node, lo;
};
__device__ __forceinline__ Row row_of(const WindowArgs& a, const Span& s, int32_t r) {
    const TreeQueries& tq = a.tq;
    const int32_t window = a.window;
    Row row{-1, 0};
    if (r >= s.rows) return row;
    row.node = (int32_t)quotient((uint32_t)r, a.by_group);
    row.lo = s.ctx - window + 1 + row.node;
    if (tq.mask && window != kNoWindow) {
        const uint32_t* words = tq.mask + (int64_t)(s.nodes.first + row.node) * tq.mask_words;
        int32_t seen = 0;
        for (int32_t w = 0; 32 * w < s.nodes.count; ++w) {
            const int32_t left = s.nodes.count - 32 * w;
            seen += __builtin_popcount(words[w] & (left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1u));
        }
        row.lo = s.ctx - window + seen;
    }
    return row;
}
// Which of the 32 keys from key0 on the row sees.
__device__ __forceinline__ uint32_t row_sees(const TreeQueries& tq, const Span& s, const Row& row, int32_t sinks, int32_t key0) {
    uint32_t near = ~below_key(row.lo, key0) | below_key(sinks, key0);
    if (!tq.mask) return row.node < 0 ? 0u : near & below_key(s.ctx + row.node + 1, key0);
    uint32_t word[1] = {row.node < 0 ? 0u : 0xFFFFFFFFu};
    if (key0 + 31 >= s.ctx) {
        seen_keys<1>(word, tq, s.nodes, s.ctx, row.node, key0);
        near |= ~below_key(s.ctx, key0);  // the mask alone decides over the nodes
    }
    return word[0] & near;
}

// ---- few rows -----------------------------------------------------------------------------------------------------

// A tile of 32 cells of 4 bits as a lane loads it: of key 16 (l / 32) + l % 16 the 32 codes of K's group l / 16 % 2, V's,
// and the scale dword.
struct Packed {
    U32x4 k, v;
    uint32_t scales;
};
template <bool FP4>
struct RawOf {
    typedef Keys T;
};
template <>
struct RawOf<true> {
    typedef Packed T;
};

// The wave's own part of LDS, through which V's codes and the scales of a packed tile reach the lanes that need them: 32
// bytes a key, every 8 keys 32 bytes apart (so that the four rows of 32 bytes that a read touches lie in banks of their
// own), then the keys' scale dwords.
constexpr int kTurnScales = 4 * 288, kTurnBytes = kTurnScales + 4 * kTile;

// Packed cells opened as K's and V's operands: K's lane has key l % 16 of each half, elements 32 (l / 16 % 2) + 16 (l / 32) +
// 8 h .., V's lane elements 4 (l % 16) .. of the keys 16 t + 4 (l / 16) + r.
// HELD: V's scales at most 2^125 (of cells that not every row sees).
template <bool HELD>
__device__ __forceinline__ void open_keys(Keys& kv, const Packed& p, uint8_t* turn, uint32_t lane) {
    const uint32_t g = lane >> 4, n16 = lane & 15u, key = 16 * (lane >> 5) + n16;
    store16(turn + key * 32 + (key >> 3) * 32 + (g & 1u) * 16, p.v);
    *reinterpret_cast<uint32_t*>(turn + kTurnScales + 4 * key) = p.scales;
    __builtin_amdgcn_wave_barrier();  // (a wave's LDS accesses keep their order)
    asm volatile("" ::: "memory");
    uint32_t v[8];
    U32x4 vs[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        vs[t] = load16(turn + kTurnScales + 64 * t + 16 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t of = 16 * t + 4 * g;  // (its key + r lies in the same 8)
            v[4 * t + r] = *reinterpret_cast<const uint16_t*>(turn + of * 32 + (of >> 3) * 32 + r * 32 + 2 * n16);
        }
    }
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
    // the halves of the wave trade dwords, so that each has both halves of the tile
    const auto k0 = __builtin_amdgcn_permlane32_swap(p.k.x, p.k.z, false, false);
    const auto k1 = __builtin_amdgcn_permlane32_swap(p.k.y, p.k.w, false, false);
    const auto ks = __builtin_amdgcn_permlane32_swap(p.scales, p.scales, false, false);
    // the scale's byte to a float's exponent; the other bits are not looked at
    const uint32_t k_turn = g & 1u ? 17u : 9u, v_turn = lane & 8u ? 1u : 25u;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const float s = __uint_as_float(__builtin_amdgcn_alignbit(ks[t], ks[t], k_turn));
        kv.k[t][0] = fp4_open(k0[t], s);
        kv.k[t][1] = fp4_open(k1[t], s);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = (&vs[i / 4].x)[i % 4];
        uint32_t s = __builtin_amdgcn_alignbit(w, w, v_turn);
        if constexpr (HELD) {
            s &= 0x7F800000u;
            s = s < kScaleHigh << 23 ? s : kScaleHigh << 23;
        }
        kv.v[i] = uint2{fp4_pair<0>(v[i], __uint_as_float(s)), fp4_pair<1>(v[i], __uint_as_float(s))};
    }
}

// One workgroup per (sequence, KV head, share); its WAVES waves hold the same rows and take the share's tiles of 32
// keys in turn, from memory through registers. The matrix products and the order of their operands are those of
// few_rows_kernel in tree_attention.hip (K's 16 packed codes of a lane are 16 neighbouring elements of d, and the queries'
// operand is loaded in that order). Several tiles of a wave are on the way while it works on one (a packed tile is 2.2 KB: one
// ahead would leave the memory waiting), and the block numbers of 32 tiles come in one load.
// First the tiles that every row sees whole, without masks; then the others, which are few: the sinks' last, those in
// which the rows' windows begin, those of the rows' own keys.
template <int R, int WAVES, bool CAP, bool FP4, bool PAGES>
__global__ __launch_bounds__(64 * WAVES, 2) void window_few_kernel(WindowArgs a, uint32_t groups) {
    extern __shared__ float smem[];
    if (blockIdx.x >= groups) {
        fill_rows(a.tq, a.fill, a.out, a.lse, blockIdx.x - groups, gridDim.x - groups);
        return;
    }
    typedef typename RawOf<FP4>::T Raw;
    // tiles of a wave in registers (8 waves: all that they have, of a short window)
    constexpr int kAhead = FP4 || WAVES == 8 ? 4 : 2;
    const PagedCache& kv = a.kv;
    const TreeQueries& tq = a.tq;
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t g = lane >> 4, n16 = lane & 15u;
    const uint32_t id = quotient(blockIdx.x, a.by_blocks), bh = quotient(id, a.by_splits);
    const int32_t row0 = (int32_t)(blockIdx.x - id * a.plan.row_blocks) * 16 * R;
    const int32_t split = (int32_t)(id - bh * a.plan.splits);
    const int32_t b = (int32_t)quotient(bh, a.by_heads), h = (int32_t)bh - b * tq.H;
    const int32_t* table = kv.tables + (int64_t)b * kv.table_stride;
    const Span s = span_of<kTile>(tq, b);
    if (row0 >= s.rows) return;
    const Keyspan span = keyspan(a, s, row0, row0 + 16 * R - 1);
    const Tiles tiles = tiles_of<kTile>(span, a.sinks);
    const int32_t share = a.plan.share, first = split * share;
    if (first >= tiles.n) return;  // (nor does the join look at such a share)
    const int32_t end = tiles.n - first < share || split == a.plan.splits - 1 ? tiles.n : first + share;
    const int32_t total = s.ctx + s.nodes.count;
    const int32_t v0 = first + (int32_t)wave;  // the wave's tiles: v0, v0 + WAVES ..
    const int32_t count = v0 < end ? (end - v0 + WAVES - 1) / WAVES : 0;

    const uint8_t* head = reinterpret_cast<const uint8_t*>(kv.cache) + (int64_t)h * kv.head_stride * (FP4 ? 1 : 2);
    const Factors f = factors<CAP>(tq);
    const uint32_t codes = kFp4Codes * kv.block_size;  // bytes of a page's K codes
    uint8_t* turn = reinterpret_cast<uint8_t*>(smem) + wave * kTurnBytes;  // FP4, until the waves join

    // The block numbers of the wave's kAhead tiles from number j on. PAGES (bf16, block_size a multiple of 16, so that half a
    // tile lies in one page): lane 2 i + t of half t of tile j + i; otherwise, at [i], of the lane's key of tile j + i.
    constexpr int kVectors = PAGES ? 1 : kAhead;
    const uint32_t own_key = FP4 ? 16 * (lane >> 5) + n16 : lane & 31u;
    struct Blocks {
        uint32_t page[kVectors];
    };
    auto key_of = [&](int32_t j, int i) {
        const int32_t v = v0 + (j + (PAGES ? (int32_t)(lane >> 1) : i)) * WAVES;
        return (uint32_t)tiles.key((v < end ? v : end - 1) * kTile) + (PAGES ? (lane & 1u) * 16 : own_key);
    };
    auto blocks_of = [&](int32_t j) {
        Blocks p;
#pragma unroll
        for (int i = 0; i < kVectors; ++i) p.page[i] = page_of(kv, table, key_of(j, i));
        return p;
    };
    // The i-th of the tiles from number j on; which of its keys there are. A cell that is not there is read from the
    // cache's first page, and masked.
    auto fetch = [&](Raw& raw, const Blocks& p, int32_t j, int i) -> uint32_t {
        const uint32_t key = key_of(j, i), blk = block_of(key, kv);
        uint32_t at = key - blk * kv.block_size, page = p.page[PAGES ? 0 : i];
        const bool is = blk < kv.table_width && page < kv.num_blocks && key < (uint32_t)total;
        const uint64_t there = __ballot(is);
        page = is ? page : 0u;
        at = is ? at : 0u;
        const uint8_t* base = head + (int64_t)page * kv.block_stride * (FP4 ? 1 : 2);
        if constexpr (FP4) {
            const uint8_t* k = base + (int64_t)(at * kFp4Codes + (g & 1u) * 16);
            raw.k = load16(k);
            raw.v = load16(k + codes);
            raw.scales = *reinterpret_cast<const uint32_t*>(base + (int64_t)(2 * codes + 4 * at));
            return (uint32_t)(there & 0xFFFFu) | (uint32_t)(there >> 16 & 0xFFFF0000u);
        } else if constexpr (PAGES) {
            const uint8_t* first_cell = base + (int64_t)at * kv.page_stride * 2;
            const uint32_t k_at = n16 * (uint32_t)kv.page_stride + 8 * g;
            const uint32_t v_at = 4 * g * (uint32_t)kv.page_stride + kHeadDim + 4 * n16;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint64_t w = (uint64_t)(uintptr_t)first_cell;
                const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)w, 2 * i + t), hi = __builtin_amdgcn_readlane((uint32_t)(w >> 32), 2 * i + t);
                const uint16_t* cells = reinterpret_cast<const uint16_t*>((uintptr_t)((uint64_t)hi << 32 | lo));
                raw.k[t][0] = load16(cells + k_at);
                raw.k[t][1] = load16(cells + k_at + 32);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    raw.v[4 * t + r] = *reinterpret_cast<const uint2*>(cells + v_at + r * (uint32_t)kv.page_stride);
            }
            return (there >> (2 * i) & 1u ? 0xFFFFu : 0u) | (there >> (2 * i + 1) & 1u ? 0xFFFF0000u : 0u);
        } else {
            // a key's cell, from the lane that holds its place
            const uint64_t cell = (uint64_t)(uintptr_t)(base + (int64_t)at * kv.page_stride * 2);
            auto of_key = [&](uint32_t k) {
                const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute((int)(k << 2), (int)(uint32_t)cell);
                const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute((int)(k << 2), (int)(uint32_t)(cell >> 32));
                return reinterpret_cast<const uint16_t*>((uintptr_t)((uint64_t)hi << 32 | lo));
            };
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint16_t* k = of_key(16 * t + n16);
                raw.k[t][0] = load16(k + 8 * g);
                raw.k[t][1] = load16(k + 32 + 8 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    raw.v[4 * t + r] = *reinterpret_cast<const uint2*>(of_key(16 * t + 4 * g + r) + kHeadDim + 4 * n16);
            }
            return (uint32_t)there;
        }
    };

    Rows<R> w;
    Row row[R];
#pragma unroll
    for (int rq = 0; rq < R; ++rq) {
        const int32_t r = row0 + 16 * rq + (int32_t)n16;
        row[rq] = row_of(a, s, r);
        w.q[rq][0] = w.q[rq][1] = U32x4{0u, 0u, 0u, 0u};
        if (row[rq].node >= 0) {
            const uint16_t* q = tq.q + (int64_t)(s.nodes.first + row[rq].node) * tq.q_rs +
                                (int64_t)(h * tq.G + r - row[rq].node * tq.G) * tq.q_hs;
            // in the order of d that K's operand has
            w.q[rq][0] = load16(q + (FP4 ? 32 * (g & 1u) + 16 * (g >> 1) : 8 * g));
            w.q[rq][1] = load16(q + (FP4 ? 32 * (g & 1u) + 16 * (g >> 1) + 8 : 32 + 8 * g));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w.o[rq][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        w.base[rq] = kNone;
        w.c[rq] = f.c;
        w.l[rq] = 0.0f;
    }

    // The tiles that every row sees whole, below whole_sinks and from `near` to `own`.
    const int2 seen_whole = whole_tiles<kTile>(span, tiles, a.sinks);
    const int32_t whole_sinks = tiles.sinks > 0 ? a.sinks / kTile : 0, near = seen_whole.x, own = seen_whole.y;
    bool left_out = false;  // such a tile with a key that is not there
    // A tile that some rows may not see whole, or with keys that are not there.
    auto masked = [&](int32_t v, const Raw& raw, uint32_t exist) {
        const int32_t key0 = tiles.key(v * kTile);
        const uint32_t there = exist & below_key(total, key0);
        if (there == 0u) return;
        uint32_t sees[R];
#pragma unroll
        for (int rq = 0; rq < R; ++rq) sees[rq] = there & row_sees(tq, s, row[rq], a.sinks, key0);
        Keys keys;
        if constexpr (FP4) {
            open_keys<true>(keys, raw, turn, lane);
            masked_tile<R, CAP>(w, keys, f.c, f.capped, sees, lane);
        } else {
            keys = raw;
            // (what lies in the places of keys that are not there may be anything)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(there >> (16 * (i / 4) + 4 * g + i % 4) & 1u)) keys.v[i] = uint2{0u, 0u};
            const bool odd = any_odd(keys);
            if (odd) {
                Keys finite = keys;
                drop_odd(finite);
                masked_tile<R, CAP>(w, finite, f.c, f.capped, sees, lane);
                add_odd<R>(w, keys, sees, lane);
            } else {
                masked_tile<R, CAP>(w, keys, f.c, f.capped, sees, lane);
            }
        }
    };
    // the wave's first tile from number v on
    auto own_from = [&](int32_t v) {
        if (v < first) v = first;
        return v + ((int32_t)wave - (v - first) % WAVES + WAVES) % WAVES;
    };
    int32_t before = own_from(whole_sinks);  // the wave's first tile that is not whole
    if (before >= near) before = own_from(own);
    if (count > 0) {
        // kAhead tiles to a round. Every load is made in every round (past the last tile, of some tile again), so that the
        // compiler knows how many are on the way and waits for the oldest alone; block numbers come two rounds ahead. The last round
        // brings nothing for a next one (in a captured graph, with such loads and without: a token behind a window of 1024 keys
        // 16.2 and 12.6 us, 64 sequences of up to 1024 packed keys 20.6 and 16.3, of 4096 33.8 and 31.5, of 16384 93.6 and
        // 98.1, 16 of 65536 98.6 and 96.8).
        // The first tile that is not whole comes behind the first round's, in the slot that is still free.
        Raw raw[kAhead];
        uint32_t there[kAhead];
        Blocks blocks = blocks_of(0), next = blocks_of(kAhead);
        const int32_t j_before = before < end ? (before - v0) / WAVES : 0;
        const Blocks blocks_before = blocks_of(j_before);
        auto bring = [&](int slot, const Blocks& from, int32_t j) {
            there[slot] = fetch(raw[slot], from, j, slot);
            __builtin_amdgcn_sched_barrier(0);  // (the tiles' loads in their order)
        };
        auto work = [&](int32_t j, Raw& cur, bool all) {
            const int32_t v = v0 + j * WAVES;
            if (j >= count || v >= own || (v < near && v >= whole_sinks)) return;
            if (!all) {
                left_out = true;
            } else if constexpr (FP4) {
                Keys keys;
                open_keys<false>(keys, cur, turn, lane);
                open_tile<R, CAP>(w, keys, f.c, f.capped);
            } else {
                open_tile<R, CAP>(w, cur, f.c, f.capped);
            }
        };
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i) bring(i, blocks, 0);
        if (before < end) {
            const uint32_t exist = fetch(raw[kAhead - 1], blocks_before, j_before, 0);
            masked(before, raw[kAhead - 1], exist);
        }
        auto round = [&](int32_t q, auto more) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (i == 0)
                    bring(kAhead - 1, blocks, q * kAhead);
                else if (decltype(more)::value)
                    bring(i - 1, next, (q + 1) * kAhead);
                work(q * kAhead + i, raw[i], there[i] == 0xFFFFFFFFu);
            }
        };
        int32_t q = 0;
#pragma unroll 1
        for (; (q + 1) * kAhead < count; ++q) {
            const Blocks after = blocks_of((q + 2) * kAhead);
            round(q, std::true_type{});
            blocks = next;
            next = after;
        }
        round(q, std::false_type{});
    }
    // The others (all tiles where some were left out, but those that are done).
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int32_t from = left_out ? (i == 0 ? 0 : tiles.n) : i == 0 ? whole_sinks : own;
        const int32_t upto = left_out ? tiles.n : i == 0 ? near : tiles.n;
        for (int32_t v = own_from(from); v < upto && v < end; v += WAVES) {
            if (v == before) continue;
            const int32_t j = (v - v0) / WAVES;
            Raw raw;
            const uint32_t exist = fetch(raw, blocks_of(j), j, 0);
            if (exist != 0xFFFFFFFFu || !(v < whole_sinks || (v >= near && v < own))) masked(v, raw, exist);
        }
    }

    // Join the waves: each leaves m's base, l and O of its rows in LDS.
    if (FP4) __syncthreads();
    float* so = smem;                          // [WAVES][16 R][kPad]
    float* sm = smem + WAVES * 16 * R * kPad;  // [WAVES][16 R]
    float* sl = sm + WAVES * 16 * R;           // [WAVES][16 R]
#pragma unroll
    for (int rq = 0; rq < R; ++rq) {
        const float l = group_sum(w.l[rq]);
        const uint32_t r = wave * 16 * R + 16 * rq + n16;
        if (g == 0) {
            sm[r] = base_of<CAP>(w.base[rq], w.c[rq], f.c);
            sl[r] = l;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4*>(so + r * kPad + 16 * g + 4 * i) =
                f32x4{w.o[rq][0][i], w.o[rq][1][i], w.o[rq][2][i], w.o[rq][3][i]};
    }
    __syncthreads();
    const int32_t heads = tq.H * tq.G;
    const int64_t rows_all = (int64_t)tq.T * heads;
    const Results to{a.out, a.lse, a.part + split * rows_all * kHeadDim,
                     a.part + (a.plan.splits * kHeadDim + 2 * split) * rows_all, a.plan.splits == 1};
    for (int32_t e = threadIdx.x; e < 16 * R * 16; e += 64 * WAVES) {
        const int32_t r = e >> 4, d = (e & 15) * 4;
        if (row0 + r >= s.rows) continue;
        float top = -__builtin_inff();
#pragma unroll
        for (int k = 0; k < WAVES; ++k) top = __builtin_fmaxf(top, sm[k * 16 * R + r]);
        const float base = top == -__builtin_inff() ? 0.0f : top;
        float l = 0.0f;
        f32x4 o{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
            const float x = exp2_hw(sm[k * 16 * R + r] - base);
            l = __builtin_fmaf(sl[k * 16 * R + r], x, l);
            const f32x4 p = *reinterpret_cast<const f32x4*>(so + (k * 16 * R + r) * kPad + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(p[i], x, o[i]);
        }
        const int32_t node = (int32_t)quotient((uint32_t)(row0 + r), a.by_group);
        put_row4(to, (int64_t)(s.nodes.first + node) * heads + h * tq.G + (row0 + r - node * tq.G), d, top, l, o);
    }
}

// ---- many rows ----------------------------------------------------------------------------------------------------

// The WAVES waves of a workgroup hold 32 rows each and share the keys, staged as bf16 in LDS 128 at a time, in two
// buffers: four threads a key bring a quarter of its cell each into registers while the waves work on the tile before, open it
// where it is packed, and leave it in the other buffer; one barrier a tile. So a key is opened once for all rows of the
// workgroup. LDS layout and matrix operands as many_rows_kernel of tree_attention.hip.
// Measured: 4 sequences of up to 65536 packed keys, 8 KV heads, 384 rows a head: 203 us, 660 TFLOP/s (with 64 keys a stage of 4 waves, so
// twice the barriers, 214); two prompts of 4096 tokens, 64 heads, window 1024: 200 us, 545 TFLOP/s. The vector unit is what is
// busiest (a score's exponential, its product, sum and rounding: of 32 x 32 scores about 60 instructions of a wave to 8 of the matrix
// cores, which take half as long); a window's short run of tiles also has its first loads and its masked ends to wait for.
constexpr int kStage = 128;
constexpr int kManyLds = 2 * kStage * (256 + 4);

// PAGES (block_size a multiple of 16, so that a wave's 16 keys lie in one page): where the cells of tiles that every row sees
// whole lie is scalar work, and a lane adds its own place in 16 cells, which is always the same (pages of 24
// cells, for which each lane works it out: 250 us for 384 rows where pages of 64 take 204, 262 for 512 rows where those take 226).
template <int WAVES, bool CAP, bool FP4, bool PAGES>
__global__ __launch_bounds__(64 * WAVES, 2) void window_many_kernel(WindowArgs a, uint32_t groups, uint32_t grid) {
    if (blockIdx.x >= grid) {
        fill_rows(a.tq, a.fill, a.out, a.lse, blockIdx.x - grid, gridDim.x - grid);
        return;
    }
    constexpr int kSubs = kStage / 32, kCells = kStage / (16 * WAVES);  // cells of a thread's in a stage, every 16 WAVES keys one
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    uint32_t* present = reinterpret_cast<uint32_t*>(lds + 2 * kStage * 256);  // [2][kStage]
    const PagedCache& kv = a.kv;
    const TreeQueries& tq = a.tq;
    const uint32_t lds0 = lds_address(lds);
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t hl = lane >> 5, n32 = lane & 31u;
    // the row blocks of one share, which read the same keys, run on one XCD next to each other
    uint32_t id = blockIdx.x, rb = 0;
    if (a.plan.row_blocks > 1) {
        const uint32_t slot = id >> 3, of = quotient(slot, a.by_blocks);
        rb = slot - of * a.plan.row_blocks;
        id = of * 8 + (id & 7u);
        if (id >= groups) return;
    }
    int32_t b, h, split, share = a.plan.share;
    if (a.plan.by_lengths) {
        const Shares r = shares_of<kStage>(tq, a.plan.groups, share, (int32_t)id, lane);
        if (r.b < 0) return;
        b = r.b, h = r.h, split = r.split, share = r.tiles;
        // for the join: each sequence's first group, its shares and their tiles
        if (rb == 0 && h == 0 && split == 0 && tid == 0) {
            a.shares[3 * b] = r.first;
            a.shares[3 * b + 1] = r.splits;
            a.shares[3 * b + 2] = r.tiles;
        }
    } else {
        const uint32_t bh = quotient(id, a.by_splits);
        split = (int32_t)(id - bh * a.plan.splits);
        b = (int32_t)quotient(bh, a.by_heads), h = (int32_t)bh - b * tq.H;
    }
    b = __builtin_amdgcn_readfirstlane(b);
    h = __builtin_amdgcn_readfirstlane(h);
    split = __builtin_amdgcn_readfirstlane(split);
    share = __builtin_amdgcn_readfirstlane(share);
    const Span s = span_of<kStage>(tq, b);
    const int32_t block0 = rb * WAVES * 32;
    if (block0 >= s.rows) return;
    const Keyspan block_span = keyspan(a, s, block0, block0 + WAVES * 32 - 1);
    const Tiles tiles = tiles_of<kStage>(block_span, a.sinks);
    const int32_t first = split * share;
    if (first >= tiles.n) return;
    const int32_t end = tiles.n - first < share || (!a.plan.by_lengths && split == a.plan.splits - 1) ? tiles.n : first + share;
    const int32_t total = s.ctx + s.nodes.count;
    const int32_t row0 = block0 + (int32_t)wave * 32;
    const bool active = row0 < s.rows;
    const Keyspan span = keyspan(a, s, row0, row0 + 31);  // of this wave's rows

    const uint8_t* head = reinterpret_cast<const uint8_t*>(kv.cache) + (int64_t)h * kv.head_stride * (FP4 ? 1 : 2);
    const int32_t* table = kv.tables + (int64_t)b * kv.table_stride;
    const Factors f = factors<CAP>(tq);

    const uint32_t codes = kFp4Codes * kv.block_size;  // bytes of a page's K codes
    // A thread's quarter (K's halves, V's halves) of its key's cell.
    const uint32_t own_key = tid >> 2, quarter = tid & 3u;
    struct Cell {
        U32x4 part[FP4 ? 1 : 4];
        uint32_t scales;
        bool there;
    } cell[kCells];
    struct Pages {
        uint32_t of[kCells];
    };
    auto key_of = [&](int32_t v, int c) {  // in tile number v
        const uint32_t key = own_key + 16 * WAVES * c;
        return (uint32_t)tiles.key(v * kStage + (int32_t)(key & ~31u)) + (key & 31u);
    };
    auto entry = [&](int32_t v) {
        Pages p;
#pragma unroll
        for (int c = 0; c < kCells; ++c) p.of[c] = page_of(kv, table, key_of(v < end ? v : end - 1, c));
        return p;
    };
    auto fetch = [&](int32_t v, const Pages& pages) {
#pragma unroll
        for (int c = 0; c < kCells; ++c) {
            // (a cell that is not there is read from the cache's first page, and dropped)
            const uint32_t key = key_of(v, c), blk = block_of(key, kv), page = pages.of[c];
            const bool is = blk < kv.table_width && page < kv.num_blocks && key < (uint32_t)total;
            const uint32_t at = is ? key - blk * kv.block_size : 0u;
            const uint8_t* base = head + (int64_t)(is ? page : 0u) * kv.block_stride * (FP4 ? 1 : 2);
            cell[c].there = is;
            if constexpr (FP4) {
                cell[c].part[0] = load16(base + (int64_t)((quarter >> 1) * codes + at * kFp4Codes + (quarter & 1u) * 16));
                cell[c].scales = *reinterpret_cast<const uint32_t*>(base + (int64_t)(2 * codes + 4 * at));
            } else {
                const uint8_t* own = base + (int64_t)at * kv.page_stride * 2 + 64 * quarter;
#pragma unroll
                for (int i = 0; i < 4; ++i) cell[c].part[i] = load16(own + 16 * i);
            }
        }
    };
    const uint32_t swizzle = quarter < 2 ? own_key & 7u : (own_key >> 1 & 1u) << 2;
    auto put = [&](int buf) {
#pragma unroll
        for (int n = 0; n < kCells; ++n) {
            Cell& c = cell[n];
            const uint32_t key = own_key + 16 * WAVES * n;  // (the swizzles are the same)
            uint8_t* at = lds + buf * (kStage * 256) + (quarter >> 1) * (kStage * 128) + key * 128;
            if (!c.there) {
#pragma unroll
                for (U32x4& x : c.part) x = U32x4{0u, 0u, 0u, 0u};
                c.scales = 0;
            }
            if constexpr (FP4) {
                uint32_t byte = c.scales >> (8 * quarter) & 0xFFu;
                if (quarter >= 2) byte = byte < kScaleHigh ? byte : kScaleHigh;  // (V: see the top)
                const float scale = __uint_as_float(byte << 23);
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                    store16(at + ((4 * (quarter & 1u) + i) ^ swizzle) * 16, fp4_open((&c.part[0].x)[i], scale));
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) store16(at + ((4 * (quarter & 1u) + i) ^ swizzle) * 16, c.part[i]);
            }
            if (quarter == 0) present[buf * kStage + key] = c.there;
        }
    };

    // This lane's places in a stage, as addresses in LDS: all that the whole tiles' loop adds to them are constants, which
    // the reads carry (worked out at every read they were a seventh of its vector instructions).
    struct Places {
        uint32_t k[4], v[2];
        __device__ __forceinline__ void move(uint32_t by) {
#pragma unroll
            for (uint32_t& x : k) x += by;
#pragma unroll
            for (uint32_t& x : v) x += by;
        }
    } places;
    {
        const uint32_t t16 = lane & 15u;
#pragma unroll
        for (int i = 0; i < 4; ++i) places.k[i] = lds0 + n32 * 128 + (((2 * i + hl) ^ (n32 & 7u)) << 4);
#pragma unroll
        for (int c = 0; c < 2; ++c)
            places.v[c] = lds0 + ((kStage * 128 + (4 * hl + (t16 >> 2)) * 128 +
                                   ((2 * (lane >> 4 & 1u) + (t16 >> 1 & 1u)) ^ (t16 >> 3) << 2) * 16 + (t16 & 1u) * 8) ^ c * 64);
    }
    auto place_of = [&](int buf, int sub) {
        Places p = places;
        p.move(buf * (kStage * 256) + sub * 4096);
        return p;
    };
    auto read_k = [&](Keys32& k, const Places& p, int sub) {
        typedef __attribute__((address_space(3))) const U32x4 Lds;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Lds* from = (Lds*)(uintptr_t)p.k[i] + 256 * sub;
            k.k[i] = U32x4{from->x, from->y, from->z, from->w};
        }
    };
    auto read_v = [&](Keys32& k, const Places& p, int sub) {
        typedef __attribute__((address_space(3))) i16x4 LdsFour;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                LdsFour* from = (LdsFour*)(uintptr_t)p.v[c] + 512 * sub + 256 * ks;
                const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(from)),
                            z = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(from + 128));
                k.v[c][ks] = U32x4{a.x, a.y, z.x, z.y};
            }
    };

    Rows32<1> w;
    const int32_t r = row0 + (int32_t)n32;
    const Row row = row_of(a, s, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) w.q[0][i] = U32x4{0u, 0u, 0u, 0u};
    if (row.node >= 0) {
        const uint16_t* q = tq.q + (int64_t)(s.nodes.first + row.node) * tq.q_rs +
                            (int64_t)(h * tq.G + r - row.node * tq.G) * tq.q_hs + 8 * hl;
#pragma unroll
        for (int i = 0; i < 4; ++i) w.q[0][i] = load16(q + 16 * i);
    }
    w.o[0][0] = w.o[0][1] = f32x16{0.f};
    w.base[0] = kNone;
    w.c[0] = f.c;
    w.l[0] = 0.0f;

    auto masked = [&](int buf, int sub, int32_t key0, uint32_t keys_there) {
        Keys32 k;
        const uint32_t sees = bits_of_scores(keys_there & row_sees(tq, s, row, a.sinks, key0), hl);
        const Places p = place_of(buf, sub);
        read_k(k, p, 0);
        read_v(k, p, 0);
        bool odd = false;  // infinities and NaN in V: see add_odd
        if constexpr (!FP4) {
            u16x2 most{0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, (&k.v[i / 8][i / 4 % 2].x)[i % 4] & 0x7FFF7FFFu));
            odd = __any(most.x >= 0x7F80 || most.y >= 0x7F80);
            if (odd) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint32_t& v = (&k.v[i / 8][i / 4 % 2].x)[i % 4];
                    v = finite_pair(v);
                }
            }
        }
        f32x16 sc;
        scores32<1>(sc, w, 0, k);
        add32<1, CAP, true>(w, 0, sc, k, f, sees);
        if (!odd) return;
        read_v(k, p, 0);
#pragma unroll 1
        for (int kind = 0; kind < 3; ++kind) {
            const float adds = kind == 0 ? __builtin_inff() : kind == 1 ? -__builtin_inff() : __builtin_nanf("");
            const uint32_t which = kind == 0 ? 0x7F80u : kind == 1 ? 0xFF80u : 0u;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f32x16 met{0.f};
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    U32x4 ones, seen;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        (&ones.x)[j] = ones_of_kind((&k.v[c][ks].x)[j], which);
                        const uint32_t two = sees >> (8 * ks + 2 * j);
                        (&seen.x)[j] = (two & 1u ? 0x3F80u : 0u) | (two & 2u ? 0x3F800000u : 0u);
                    }
                    met = mfma32(ones, seen, met);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (met[i] > 0.0f) w.o[0][c][i] += adds;
            }
        }
    };
    // A tile that is not whole, or of which keys may not be there.
    auto partial = [&](int32_t v, int buf) {
        uint64_t exists[kStage / 64];
        bool all = true;
#pragma unroll
        for (int i = 0; i < kStage / 64; ++i) {
            exists[i] = __ballot(present[buf * kStage + 64 * i + lane] != 0u);
            all &= exists[i] == ~0ull;
        }
        // the 32s that all the wave's rows see whole (but some of the sinks alone), from `from` to `upto`, with every key
        // there; then the others
        const int2 of_rows = whole_tiles<32>(span, tiles, a.sinks);
        int32_t from = of_rows.x - v * kSubs, upto = of_rows.y - v * kSubs;
        if (from < 0) from = 0;
        if (upto > kSubs) upto = kSubs;
        if (!all || from >= upto) from = upto = 0;
        if (from < upto) {
            Keys32 k;
            f32x16 sc[2];
            Places p = place_of(buf, from);
            read_k(k, p, 0);
            scores32<1>(sc[0], w, 0, k);
            auto step = [&](int32_t sub, f32x16& own, f32x16& next) {
                read_v(k, p, 0);
                if (sub + 1 < upto) {
                    read_k(k, p, 1);
                    scores32<1>(next, w, 0, k);
                }
                p.move(4096);
                add32<1, CAP, false>(w, 0, own, k, f, 0u);
            };
#pragma unroll 1
            for (int32_t sub = from;;) {
                step(sub, sc[0], sc[1]);
                if (++sub >= upto) break;
                step(sub, sc[1], sc[0]);
                if (++sub >= upto) break;
            }
        }
#pragma unroll 1
        for (int32_t sub = 0; sub < kSubs; ++sub) {
            if (sub >= from && sub < upto) continue;
            const uint32_t keys_there = (uint32_t)((kStage > 64 && sub & 2 ? exists[kStage / 64 - 1] : exists[0]) >> (32 * (sub & 1)));
            const int32_t at = tiles.key(v * kStage + 32 * sub);
            if (may_be_seen(span, a.sinks, at) && keys_there != 0u) masked(buf, sub, at, keys_there);
        }
    };

    // First the tiles that every row of the workgroup sees whole, up to the first whose blocks are not all there: nobody
    // asks for single rows or keys in them. Then those before, and those behind.
    const int2 block_whole = whole_tiles<kStage>(block_span, tiles, a.sinks);
    int32_t whole0 = block_whole.x < first ? first : block_whole.x > end ? end : block_whole.x;
    const int32_t whole1 = block_whole.y > end ? end : block_whole.y < whole0 ? whole0 : block_whole.y;
    int32_t whole = whole1 - whole0;
    const int32_t count = end - first;
    auto number = [&](int32_t i) {  // of the i-th tile
        if (i < whole) return whole0 + i;
        return i - whole < whole0 - first ? first + i - whole : first + i;
    };
    // The tile after the next one's block numbers are on the way before the next one's cells, so that nobody waits for
    // these with those.
    Pages page = entry(number(0)), after = entry(number(1));
    auto bring = [&](int32_t i) {
        page = after;
        after = entry(number(i + 1));
        if (i < count) fetch(number(i), page);
    };
    fetch(number(0), page);
    if (whole > 0) {
        // Are their blocks there? Every wave looks at all of them, 64 a load, four loads on the way. (A share of 257 tiles in 2050
        // blocks of 16 takes as long as in 513 of 64: 32 sequences of 48 nodes over up to 32768 packed keys 797 and 786 us, against
        // 1568 with places worked out per lane and key.)
        const uint32_t block = block_of((uint32_t)tiles.key(whole0 * kStage), kv);
        const uint32_t blocks = block_of((uint32_t)tiles.key((whole0 + whole) * kStage - 32) + 31, kv) - block + 1;
        uint32_t gone = 0;  // from the lane's first block that is not there on
#pragma unroll 4
        for (uint32_t i = lane; i < blocks; i += 64) {
            const uint32_t n = block + i, page = (uint32_t)table[n < kv.table_width ? n : kv.table_width - 1];
            if (!(n < kv.table_width && page < kv.num_blocks) && gone == 0) gone = blocks - i;
        }
        if (__any(gone != 0)) {
            const int64_t left = (int64_t)(block + blocks - wave_most(gone)) * kv.block_size - tiles.key(whole0 * kStage);
            whole = left < kStage ? 0 : (int32_t)(left / kStage);
            fetch(number(0), entry(number(0)));
            after = entry(number(1));
        }
    }
    put(0);
    __syncthreads();
    if (whole > 0) {
        // Where the whole tiles' keys come from and go to (PAGES): the wave's first key of tile i, a lane's place in 16 cells and in
        // a stage. Such keys are there, and V's scales need not be held.
        const int32_t key0 = __builtin_amdgcn_readfirstlane(tiles.key(whole0 * kStage) + 16 * (int32_t)wave);
        const uint32_t in16 = lane >> 2, own = FP4 ? in16 * kFp4Codes + (quarter >> 1) * codes + (quarter & 1u) * 16
                                                   : in16 * 2 * (uint32_t)kv.page_stride + 64 * quarter;
        uint32_t put_at[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            put_at[i] = lds0 + (quarter >> 1) * (kStage * 128) + own_key * 128 + ((4 * (quarter & 1u) + i) ^ swizzle) * 16;
        auto whole_entry = [&](int32_t i) {
            Pages p;
#pragma unroll
            for (int c = 0; c < kCells; ++c) p.of[c] = (uint32_t)table[quotient((uint32_t)(key0 + i * kStage + 16 * WAVES * c), a.by_block)];
            return p;
        };
        auto whole_fetch = [&](int32_t i, const Pages& pages) {
#pragma unroll
            for (int c = 0; c < kCells; ++c) {
                const uint32_t key = (uint32_t)(key0 + i * kStage + 16 * WAVES * c);
                const uint32_t cell_at = key - quotient(key, a.by_block) * kv.block_size;
                const uint32_t page = __builtin_amdgcn_readfirstlane(pages.of[c]);
                const uint8_t* base = head + (int64_t)page * kv.block_stride * (FP4 ? 1 : 2);
                if constexpr (FP4) {
                    cell[c].part[0] = load16(base + cell_at * kFp4Codes + own);
                    cell[c].scales = *reinterpret_cast<const uint32_t*>(base + 2 * codes + 4 * cell_at + 4 * in16);
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n) cell[c].part[n] = load16(base + (int64_t)cell_at * kv.page_stride * 2 + own + 16 * n);
                }
            }
        };
        auto whole_put = [&](int buf) {
            typedef __attribute__((address_space(3))) U32x4 Lds;
#pragma unroll
            for (int c = 0; c < kCells; ++c) {
                const float scale = __uint_as_float(__builtin_amdgcn_alignbit(cell[c].scales, cell[c].scales, 8 * quarter + 9));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const U32x4 v = FP4 ? fp4_open((&cell[c].part[0].x)[i], scale) : cell[c].part[FP4 ? 0 : i];
                    Lds* to = (Lds*)(uintptr_t)(put_at[i] + buf * (kStage * 256)) + 128 * WAVES * c;
                    to->x = v.x, to->y = v.y, to->z = v.z, to->w = v.w;
                }
            }
        };
        // add32 for them, its products in the order in which neighbours do not wait for each other.
        auto add_whole = [&](f32x16& s, const Keys32& k) {
            U32x4 pb[2];
            float sum = weights32<CAP, false>(s, w.base[0], CAP ? f.c : w.c[0], f.capped, 0u, pb);
            if (__any(!(sum <= kMost))) {
                raise32<1, CAP>(w, 0, s, f.c, f.capped);
                sum = weights32<CAP, false>(s, w.base[0], CAP ? f.c : w.c[0], f.capped, 0u, pb);
            }
            w.l[0] += sum;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int c = 0; c < 2; ++c) w.o[0][c] = mfma32(k.v[c][ks], pb[ks], w.o[0][c]);
        };
        // One 32 keys' scores are on the way in the matrix cores while the vector unit takes the last ones' exponentials,
        // over the barrier too: a tile's last weights are taken behind it, with the next one's first scores on the way.
        // The stage's last part goes ahead of the other workgroup's waves, so that this one's reach their barrier together; the
        // phases are kept apart (trees of 48 nodes over 65536 packed keys, 64 a stage: 214 us; with the phases mixed by the compiler, which
        // then puts matrix instructions behind each other, 274).
        Keys32 k;
        f32x16 sc[2];
        if (active) {
            read_k(k, places, 0);
            scores32<1>(sc[0], w, 0, k);
        }
        Places p = places;
        auto tile = [&](int32_t i, auto inner) {  // inner: the next one is such a tile too, and its cells are PAGES'
            constexpr bool kInner = decltype(inner)::value;
            const int buf = i & 1;
            if constexpr (kInner) {
                page = after;
                after = i + 2 < whole ? whole_entry(i + 2) : entry(number(i + 2));
                whole_fetch(i + 1, page);
            } else {
                bring(i + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (active) {
#pragma unroll
                for (int sub = 0; sub < kSubs; ++sub) {
                    read_v(k, p, sub);
                    if (sub + 1 < kSubs) {
                        read_k(k, p, sub + 1);
                        scores32<1>(sc[(sub + 1) % 2], w, 0, k);
                        add_whole(sc[sub % 2], k);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);
            if constexpr (kInner)
                whole_put(buf ^ 1);  // (nobody reads it since the last barrier)
            else if (i + 1 < count)
                put(buf ^ 1);
            __syncthreads();
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
            p.move(buf ? -(kStage * 256) : kStage * 256);
            if (active) {
                if (kInner || i + 1 < whole) {
                    read_k(k, p, 0);
                    scores32<1>(sc[0], w, 0, k);
                }
                add_whole(sc[1], k);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        int32_t i = 0;
        if constexpr (PAGES) {
#pragma unroll 1
            for (; i + 1 < whole; ++i) tile(i, std::true_type{});
        }
#pragma unroll 1
        for (; i < whole; ++i) tile(i, std::false_type{});
    }
#pragma unroll 1
    for (int32_t i = whole; i < count; ++i) {
        bring(i + 1);
        if (active) partial(number(i), i & 1);
        if (i + 1 < count) {
            put((i & 1) ^ 1);
            __syncthreads();
        }
    }
    if (!active) return;
    const int32_t heads = tq.H * tq.G;
    constexpr int kRows = WAVES * 32;
    const int64_t part0 = ((int64_t)id * a.plan.row_blocks + rb) * kRows - block0;
    const Results to{a.out, a.lse, a.part, a.part + (int64_t)a.plan.groups * a.plan.row_blocks * kRows * kHeadDim, a.plan.splits == 1};
    const float l = w.l[0] + lane_xor<32>(w.l[0]);
    const float top = base_of<CAP>(w.base[0], w.c[0], f.c);
    if (row.node < 0) return;
    const int64_t at = to.whole ? (int64_t)(s.nodes.first + row.node) * heads + h * tq.G + r - row.node * tq.G : part0 + r;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            put_row4(to, at, 32 * c + 8 * i + 4 * (int32_t)hl, top, l,
                     f32x4{w.o[0][c][4 * i], w.o[0][c][4 * i + 1], w.o[0][c][4 * i + 2], w.o[0][c][4 * i + 3]});
}

// The shares of a row joined: 16 lanes a row, 4 elements of d a lane, eight shares' loads on the way at a time.
__global__ __launch_bounds__(256) void window_join_kernel(WindowArgs a) {
    const TreeQueries& tq = a.tq;
    const int32_t heads = tq.H * tq.G;
    const int32_t row = blockIdx.x * 16 + (int32_t)(threadIdx.x >> 4), d = 4 * (int32_t)(threadIdx.x & 15u);
    const int32_t b = blockIdx.y;
    const Span s = span_of<kTile>(tq, b);
    if (row >= s.nodes.count * heads) return;
    // the row's block, its tiles as the attending workgroup counted them, its first share's place
    const int32_t node = row / heads, hq = row - node * heads, h = (int32_t)quotient((uint32_t)hq, a.by_group), r = node * tq.G + hq - h * tq.G;
    const int64_t at = (int64_t)s.nodes.first * heads + row;
    int32_t splits;
    int64_t from, step, all;
    if (a.plan.many) {
        const int32_t rows = 32 * a.plan.waves, block0 = r / rows * rows;
        const Keyspan span = keyspan(a, s, block0, block0 + rows - 1);
        const int32_t n = tiles_of<kStage>(span, a.sinks).n;
        int32_t group = b * tq.H * a.plan.splits, of_head = a.plan.splits, share = a.plan.share;
        if (a.plan.by_lengths) group = a.shares[3 * b], of_head = a.shares[3 * b + 1], share = a.shares[3 * b + 2];
        splits = (n + share - 1) / share;  // (a chain's first rows may end before the sequence's last share)
        if (!a.plan.by_lengths && splits > a.plan.splits) splits = a.plan.splits;
        step = (int64_t)a.plan.row_blocks * rows;
        from = (int64_t)(group + h * of_head) * step + r;
        all = a.plan.groups * step;
    } else {
        const int32_t n = tiles_of<kTile>(keyspan(a, s, 0, s.rows - 1), a.sinks).n;
        splits = (n + a.plan.share - 1) / a.plan.share;
        if (splits > a.plan.splits) splits = a.plan.splits;
        step = (int64_t)tq.T * heads;
        from = at;
        all = a.plan.splits * step;
    }
    const float* po = a.part + from * kHeadDim + d;
    const float* pm = a.part + all * kHeadDim + from * 2;
    float base = -__builtin_inff(), l = 0.0f;  // the largest base so far
    f32x4 o{0.f, 0.f, 0.f, 0.f};
    constexpr int kAtOnce = 8;
    for (int32_t s0 = 0; s0 < splits; s0 += kAtOnce) {
        f32x4 p[kAtOnce];
        float2 ml[kAtOnce];
        float top = base;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t k = s0 + j < splits ? s0 + j : s0;
            p[j] = *reinterpret_cast<const f32x4*>(po + k * step * kHeadDim);
            ml[j] = *reinterpret_cast<const float2*>(pm + k * step * 2);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) top = __builtin_fmaxf(top, ml[j].x);  // (a repeated one changes nothing)
        const float ref = top == -__builtin_inff() ? 0.0f : top;
        const float keep = exp2_hw(base - ref);
        l *= keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= keep;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (s0 + j >= splits) break;
            const float x = exp2_hw(ml[j].x - ref);
            l = __builtin_fmaf(ml[j].y, x, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(p[j][i], x, o[i]);
        }
        base = top;
    }
    put_row4(Results{a.out, a.lse, nullptr, nullptr, true}, at, d, base, l, o);
}

__global__ __launch_bounds__(256) void window_fill_kernel(TreeQueries tq, uint32_t fill, uint16_t* __restrict__ out,
                                                          float* __restrict__ lse) {
    fill_rows(tq, fill, out, lse, blockIdx.x, gridDim.x);
}
// Workgroups that fill: one to 64 KiB of all rows, 1 to 1024.
uint32_t fill_groups(const WindowArgs& a) {
    if (a.fill == 0u) return 0u;
    const int64_t n = ((int64_t)a.tq.T * a.tq.H * a.tq.G * (2 * kHeadDim + 4) + 65535) / 65536;
    return (uint32_t)(n < 1024 ? n : 1024);
}

// Do 16 neighbouring keys lie in one page, with 32-bit offsets between its rows?
bool in_pages(const WindowArgs& a, bool fp4) { return a.kv.block_size % 16 == 0 && (fp4 || a.kv.page_stride < (1 << 24)); }

template <int R, int WAVES, bool FP4>
void launch_few(const WindowArgs& a, hipStream_t stream) {
    constexpr int kLds = WAVES * 16 * R * (kPad + 2) * 4;
    static_assert(kLds <= 65536, "above, the limit would have to be raised");
    static_assert(kTurnBytes <= 16 * R * (kPad + 2) * 4, "a wave's packed tile fits its part of the join's");
    const uint32_t groups = (uint32_t)a.tq.B * a.tq.H * a.plan.splits * a.plan.row_blocks;
    const dim3 grid(groups + fill_groups(a)), block(64 * WAVES);
    const bool pages = !FP4 && in_pages(a, FP4);
    auto kernel = a.tq.softcap > 0.0f
                      ? (pages ? window_few_kernel<R, WAVES, true, FP4, !FP4> : window_few_kernel<R, WAVES, true, FP4, false>)
                      : (pages ? window_few_kernel<R, WAVES, false, FP4, !FP4> : window_few_kernel<R, WAVES, false, FP4, false>);
    hipLaunchKernelGGL(kernel, grid, block, kLds, stream, a, groups);
}

template <int WAVES, bool CAP, bool FP4, bool PAGES>
int launch_many(const WindowArgs& a, hipStream_t stream) {
    const uint32_t groups = (uint32_t)a.plan.groups;
    const uint32_t grid = a.plan.row_blocks > 1 ? (groups + 7) / 8 * 8 * a.plan.row_blocks : groups;
    auto kernel = window_many_kernel<WAVES, CAP, FP4, PAGES>;
    static std::atomic<int> done[64] = {};
    if (raise_lds_limit(reinterpret_cast<const void*>(kernel), kManyLds, done) != 0) return -1;
    hipLaunchKernelGGL(kernel, dim3(grid + fill_groups(a)), dim3(64 * WAVES), kManyLds, stream, a, groups, grid);
    return 0;
}
template <int WAVES, bool FP4>
int launch_many(const WindowArgs& a, hipStream_t stream) {
    if (in_pages(a, FP4))
        return a.tq.softcap > 0.0f ? launch_many<WAVES, true, FP4, true>(a, stream) : launch_many<WAVES, false, FP4, true>(a, stream);
    return a.tq.softcap > 0.0f ? launch_many<WAVES, true, FP4, false>(a, stream) : launch_many<WAVES, false, FP4, false>(a, stream);
}

template <bool FP4>
int launch(const WindowArgs& a, hipStream_t stream) {
    if (a.plan.many) return a.plan.waves == 8 ? launch_many<8, FP4>(a, stream) : launch_many<4, FP4>(a, stream);
    if (a.plan.waves == 8)
        launch_few<1, 8, FP4>(a, stream);
    else
        a.plan.q_tiles == 1 ? launch_few<1, 4, FP4>(a, stream) : launch_few<2, 4, FP4>(a, stream);
    return 0;
}

}  // namespace

WindowPlan plan_window_attention(int32_t B, int32_t H, int32_t G, int32_t max_nodes, int64_t max_ctx, int32_t window,
                                 int32_t sinks, int32_t num_cus) {
    WindowPlan p{};
    const int64_t rows = (int64_t)max_nodes * G, base = (int64_t)B * H;
    const bool ragged = window == kNoWindow;  // lengths that differ as the contexts do; over a window they are about equal
    p.many = rows > 32;
    // (512 rows over contexts of up to 65536 packed keys 226 us; in blocks of 128 rows, which open each key twice as often, 258; a
    // prompt of 8192 tokens behind a window of 2048 370 and 380; but two prompts of 4096 behind 1024 196 and 183)
    p.waves = p.many && rows > 128 ? 8 : 4;
    // waves without rows are idle: blocks of 128 rows where those of 256 would be filled to less than four fifths as much
    if (p.waves == 8 && 4 * ((rows + 255) / 256 * 256) > 5 * ((rows + 127) / 128 * 128)) p.waves = 4;
    p.q_tiles = rows <= 16 ? 1 : 2;
    const int64_t block_rows = p.many ? 32 * p.waves : rows, keys = p.many ? kStage : kTile;
    p.row_blocks = p.many ? (int32_t)((rows + block_rows - 1) / block_rows) : 1;
    // the tiles that a block of rows looks at (a tree's last share takes what there are more)
    int64_t tiles = (max_ctx + max_nodes + keys - 1) / keys;
    const int64_t nodes = block_rows / G + 1 < max_nodes ? block_rows / G + 1 : max_nodes;
    const int64_t near = ((int64_t)sinks + 31 + window + nodes + 31) / keys + 1;
    if (near < tiles) tiles = near;
    p.splits = 1;
    p.share = (int32_t)tiles;
    int64_t splits, most;
    if (p.many) {
        const int64_t at_once = num_cus * (p.waves == 8 ? 1 : 2), groups = base * p.row_blocks;
        p.groups = (int32_t)base;
        if (ragged && B <= 512 && base * tiles < (int64_t)1 << 31) {
            // shares by the lengths (counted in 32 bits), in one or two rounds of what the chip holds at once
            const int64_t round = at_once / p.row_blocks, rounds = round >= 2 * base ? 1 : 2;
            if (rounds * round >= 2 * base && tiles > 4) {
                p.by_lengths = true;
                p.groups = (int32_t)(rounds * round);
                p.splits = 2;  // (or more)
                p.share = 4;   // at least
            }
            return p;
        }
        // until there is twice what the chip holds at once, of at least 4 tiles
        splits = groups >= at_once ? 1 : (2 * at_once + groups - 1) / groups;
        most = tiles / 4;
    } else {
        if (tiles <= 64 && p.q_tiles * base <= num_cus) {
            // short and few: no second launch, and 16 rows a workgroup, whose waves then have room for all their tiles
            p.waves = 8;
            p.row_blocks = p.q_tiles;
            p.q_tiles = 1;
            return p;
        }
        // until there are several workgroups per CU, each of at least 4 tiles a wave: over a window, of about equal lengths, 2;
        // over contexts, more than run at once, which evens out ragged lengths
        splits = ((ragged ? 6 : 2) * num_cus + base - 1) / base;
        most = tiles / (4 * p.waves);
    }
    if (splits > most) splits = most;
    if (splits > 1) {
        p.share = (int32_t)((tiles + splits - 1) / splits);
        p.splits = (int32_t)((tiles + p.share - 1) / p.share);
    }
    if (p.many) p.groups = (int32_t)(base * p.splits);
    return p;
}

// The partial sums' rows, and of shares by the lengths each sequence's first group, shares and tiles of one.
int64_t window_attention_workspace(const WindowPlan& p, int64_t T, int64_t heads, int32_t B) {
    if (p.splits == 1) return 0;
    const int64_t rows = p.many ? (int64_t)p.groups * p.row_blocks * 32 * p.waves : p.splits * T * heads;
    return rows * (kHeadDim + 2) * 4 + (p.by_lengths ? (int64_t)B * 3 * 4 : 0);
}

int launch_window_attention(const WindowArgs& args, hipStream_t stream) {
    WindowArgs a = args;
    a.by_group = div_by((uint32_t)a.tq.G), a.by_heads = div_by((uint32_t)a.tq.H);
    a.by_block = div_by(a.kv.block_size);
    a.by_splits = div_by((uint32_t)a.plan.splits), a.by_blocks = div_by((uint32_t)a.plan.row_blocks);
    if (a.tq.B == 0) {
        hipLaunchKernelGGL(window_fill_kernel, dim3(fill_groups(a)), dim3(256), 0, stream, a.tq, a.fill, a.out, a.lse);
        return hipGetLastError() == hipSuccess ? 0 : -1;
    }
    if (int rc = a.fp4 ? launch<true>(a, stream) : launch<false>(a, stream)) return rc;
    if (a.plan.splits > 1) {
        const dim3 grid((uint32_t)(((int64_t)a.tq.max_nodes * a.tq.H * a.tq.G + 15) / 16), (uint32_t)a.tq.B);
        hipLaunchKernelGGL(window_join_kernel, grid, dim3(256), 0, stream, a);
    }
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
