// Attention of drafted tokens over the paged cache.
//
// s_ij = scale q_i . k_j (capped: cap tanh(s / cap)), p = softmax over the
// keys that node i sees, out_i = sum_j p_ij v_j, lse_i = log sum_j e^(s_ij).
// A sequence's keys are its context, which every node sees, and its nodes,
// seen as the tree mask says.
//
// One pass over the keys with a running reference m (near the row's maximum)
// and sum l per query row; rows = nodes x the query heads of one KV head, so
// every cached byte is fetched once for all of them. S^T = K Q^T takes K as it
// lies as the A operand, and O^T += V^T P^T takes P^T from the lanes that hold the
// scores: a row's statistics and its column of O^T live in the lanes with its
// scores, and P never leaves registers. P is rounded to bf16 for the second
// product (relative 2^-8 at most each, independent between keys, so the error
// of the sum stays near the bf16 output's own rounding); m, l, O and the scores
// are FP32. m moves only when a lane's weights of a tile sum to more than 2^8 (the
// lanes vote): between, p, l and O grow by up to that factor, which FP32 and bf16
// hold at full precision, and no lane waits for another's maximum.
//
// Up to 32 rows (few_rows_kernel) the cache's bytes bound it: K and V go from
// memory to the matrix core through registers, each wave its own tiles of 32
// keys. More rows (many_rows_kernel) are bound by the vector unit (the
// exponentials and what feeds the matrix instructions) and the matrix cores, which mostly take turns: keys are staged in LDS
// and shared by a workgroup's waves, 32 or 64 rows each.
#include "../../include/nrc.h"
#include "attention_core.h"
#include "cache_ops.h"
#include "kernels.h"

namespace nrc {
namespace {

// How many workgroups fill: one to 64 KiB of all rows, 1 to 1024. They run on CUs that have nothing else to do, or behind the
// others: one token of one sequence 10.0 -> 10.2 us, in 1024 rows of 64 heads 11.3, in 16384 19; 64 sequences of up to 8192
// keys 137.0 -> 137.3. (By the attending workgroups beside their work 10.5, 20.3, 133 and 138.0.)
uint32_t fill_groups(const TreeAttentionArgs& a) {
    if (a.fill == 0u) return 0u;
    const int64_t n = ((int64_t)a.tq.T * a.tq.H * a.tq.G * (2 * kHeadDim + 4) + 65535) / 65536;
    return (uint32_t)(n < 1024 ? n : 1024);
}

// The filling alone, of a call without a sequence.
__global__ __launch_bounds__(256) void fill_rows_kernel(TreeQueries tq, uint32_t fill, uint16_t* __restrict__ out,
                                                        float* __restrict__ lse) {
    fill_rows(tq, fill, out, lse, blockIdx.x, gridDim.x);
}

// Few rows (up to 16 R, R <= 2): one workgroup per (sequence, KV head,
// split); its WAVES waves hold the same rows and take the split's tiles in turn, and
// join their sums in LDS. A tile is 32 keys by 16 R rows:
//   S^T = K Q^T   4 v_mfma_f32_16x16x32_bf16 a query tile; K's lane: key l % 16, 8
//                 elements of d, straight from memory. A lane then holds, for
//                 query row l % 16, the keys 4 (l / 16) + r of both halves.
//   O^T += V^T P^T  4 more. P^T's lane needs 8 keys of query row l % 16: the
//                 ones it holds, when slot 8 g + 4 t + r of the sum stands for
//                 key 16 t + 4 g + r. V's lane loads those same 8 keys, 4 elements of
//                 d each (8 bytes), and 16 byte permutes turn them into the 4
//                 operands (operand c: d = 4 (l % 16) + c).
// Bound by the cache's bytes: a wave keeps the next tile's K and V on the way
// while it works on one, the tile after that's block numbers too (64 sequences of
// up to 8192 keys, 8 heads: 685 MB in 137 us, 5.0 TB/s, a copy reaches 5.2).
// PAGE16 (block_size a multiple of 16, page rows near each other): the 16
// keys of half a tile lie in one page, so a tile's two bases are scalars.
// Two workgroups of 4 waves a CU, as the splits are planned: R 2 keeps to half the registers for it (32 rows over
// 30000 keys of 4 sequences, 8 heads: 62 -> 42 us); a third of R 1 would leave other CUs short.
template <int R, int WAVES, bool CAP, bool PAGE16>
__global__ __launch_bounds__(64 * WAVES, R == 2 ? 2 : 1) void few_rows_kernel(PagedCache kv, TreeQueries tq, AttentionPlan plan,
                                                              uint16_t* __restrict__ out, float* __restrict__ lse,
                                                              float* __restrict__ part, uint32_t groups, uint32_t fill) {
    extern __shared__ float smem[];
    if (blockIdx.x >= groups) {
        fill_rows(tq, fill, out, lse, blockIdx.x - groups, gridDim.x - groups);
        return;
    }
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t g = lane >> 4, n16 = lane & 15u;
    const int32_t split = blockIdx.x % plan.splits;
    const uint32_t bh = blockIdx.x / plan.splits;
    const int32_t h = bh % tq.H, b = bh / tq.H;
    const int32_t* table = kv.tables + (int64_t)b * kv.table_stride;
    const int32_t first = split * plan.split_tiles;
    int32_t t = first + (int32_t)wave;
    // the first two tiles' table entries on the way before the lengths are known (key numbers stay below 2^32)
    const uint32_t page0 = page_of(kv, table, (uint32_t)t * kTile + (lane & (kTile - 1)));
    const uint32_t page1 = page_of(kv, table, (uint32_t)(t + WAVES) * kTile + (lane & (kTile - 1)));
    const Span s = span_of<kTile>(tq, b);
    if (s.rows == 0 || first >= s.all_tiles) return;  // (nor does the join look at such a split)
    int32_t end = first + plan.split_tiles;
    const int32_t last = last_tile<kTile>(tq, s, 16 * R - 1);
    if (end > last) end = last;
    const int32_t ctx_full = s.ctx / kTile;

    const uint16_t* head = kv.cache + (int64_t)h * kv.head_stride;
    const Factors f = factors<CAP>(tq);
    auto in_tile = [&](int32_t t) { return t < end && lane < kTile && lane < keys_from<kTile>(s, t); };
    auto offsets = [&](int32_t t) -> int64_t {
        return in_tile(t) ? key_offset(kv, table, (uint32_t)t * kTile + lane) : -1;
    };
    auto offsets_by = [&](int32_t t, uint32_t page) -> int64_t {
        return in_tile(t) ? key_offset(kv, (uint32_t)t * kTile + lane, page) : -1;
    };
    // a whole tile of context, every key there
    auto whole = [&](int32_t t, int64_t off) { return t < end && t < ctx_full && (uint32_t)__ballot(off >= 0) == 0xFFFFFFFFu; };
    const uint32_t k_at = n16 * (uint32_t)kv.page_stride + 8 * g, v_at = 4 * g * (uint32_t)kv.page_stride + kHeadDim + 4 * n16;
    auto fetch = [&](Keys& k, int64_t off) {
        if constexpr (PAGE16) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)off, 16 * t);
                const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)((uint64_t)off >> 32), 16 * t);
                const uint16_t* page = head + (int64_t)((uint64_t)hi << 32 | lo);
                k.k[t][0] = load16(page + k_at);
                k.k[t][1] = load16(page + k_at + 32);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    k.v[4 * t + r] = *reinterpret_cast<const uint2*>(page + v_at + r * (uint32_t)kv.page_stride);
            }
        } else {
            load_keys(k, head, off, lane);
        }
    };

    Rows<R> w;
    int32_t node[R];
    uint32_t seen[R];
    const int32_t full_end = end < ctx_full ? end : ctx_full;
    bool left_out = false;  // a tile of the context with a key that is not there
    {
        // the tiles whose every key is there and seen by all
        Keys keys[2];
        int64_t off = offsets_by(t, page0), off1 = offsets_by(t + WAVES, page1);
        bool cur_whole = whole(t, off);
        if (cur_whole) fetch(keys[0], off);
        load_rows<R>(w, node, tq, s, h, 0, lane, f.c);
        auto step = [&](Keys& cur, Keys& next) {
            const bool next_whole = whole(t + WAVES, off1);
            if (next_whole) fetch(next, off1);
            off1 = offsets(t + 2 * WAVES);
            if (cur_whole)
                open_tile<R, CAP>(w, cur, f.c, f.capped);
            else
                left_out = true;
            cur_whole = next_whole;
            t += WAVES;
        };
        while (t < full_end) {
            step(keys[0], keys[1]);
            if (t >= full_end) break;
            step(keys[1], keys[0]);
        }
    }
    // the others: the context's last, the nodes', those left out
    for (t = left_out ? first + (int32_t)wave : t; t < end; t += WAVES) {
        const int64_t off = offsets(t);
        if (whole(t, off)) continue;
        Keys keys;
        load_keys(keys, head, off, lane);
        seen_rows<R>(seen, node, (uint32_t)__ballot(off >= 0), tq, s, t * kTile);
        const bool odd = (t + 1) * kTile > s.ctx && any_odd(keys);
        if (odd) drop_odd(keys);
        masked_tile<R, CAP>(w, keys, f.c, f.capped, seen, lane);
        if (odd) {
            load_keys(keys, head, off, lane);
            add_odd<R>(w, keys, seen, lane);
        }
    }

    // Join the waves: each leaves m's base, l and O of its rows in LDS.
    float* so = smem;                          // [WAVES][16 R][kPad]
    float* sm = smem + WAVES * 16 * R * kPad;  // [WAVES][16 R]
    float* sl = sm + WAVES * 16 * R;           // [WAVES][16 R]
#pragma unroll
    for (int rq = 0; rq < R; ++rq) {
        const float l = group_sum(w.l[rq]);
        const uint32_t row = wave * 16 * R + 16 * rq + n16;
        if (g == 0) {
            sm[row] = base_of<CAP>(w.base[rq], w.c[rq], f.c);
            sl[row] = l;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
            *reinterpret_cast<f32x4*>(so + row * kPad + 16 * g + 4 * r) =
                f32x4{w.o[rq][0][r], w.o[rq][1][r], w.o[rq][2][r], w.o[rq][3][r]};
    }
    __syncthreads();
    const int32_t heads = tq.H * tq.G;
    const int64_t rows_all = (int64_t)tq.T * heads;
    const Results to{out, lse, part + split * rows_all * kHeadDim,
                     part + (plan.splits * kHeadDim + 2 * split) * rows_all, plan.splits == 1};
    for (int32_t e = threadIdx.x; e < 16 * R * 16; e += 64 * WAVES) {
        const int32_t r = e >> 4, d = (e & 15) * 4;
        if (r >= s.rows) continue;
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
        const int32_t node_r = r / tq.G;
        put_row4(to, (int64_t)(s.nodes.first + node_r) * heads + h * tq.G + (r - node_r * tq.G), d, top, l, o);
    }
}

// Many rows: the WAVES waves of a workgroup hold 32 R rows each and share the
// keys, staged in LDS kStage at a time in four buffers (of two workgroups a CU, two
// each): while the waves work on one tile the next ones come in (global_load_lds, no
// registers), and one barrier a tile. Bound by what the vector unit issues and, uncapped, by the matrix cores in turn: a
// matrix instruction takes it 8 cycles and keeps the matrix core 32, an
// exponential takes 8, other operations 4; of 32 keys and 32 rows that is 8, 16 and
// about 50. Measured: 620 TFLOP/s (4 sequences of 32768 keys, 8 heads, 512 rows
// a head: 221 us; a large matrix product 1212), 490 with a softcap (an
// exponential and a reciprocal more a score). By counters the vector unit is busy 65% of that time and the matrix
// cores 36%, with a softcap 81% and 26%. Short shares are bound by their
// loads' latency one after the other: lengths, block numbers, keys, masks.
// LDS: K rows of 128 bytes whose 16-byte chunk c lies at c ^ (key & 7), so
// that 8 lanes reading one chunk of 8 keys meet all banks; V rows with c at
// c ^ 4 in every second pair of keys, so that the 4 keys and 64 bytes that half a wave
// reads meet all banks. V's operands come by ds_read_b64_tr_b16: 16 lanes read 4
// keys of 16 elements and each gets the 4 keys of its element.
// The row blocks of one split, which read the same keys, run on one XCD next
// to each other (workgroup i runs on XCD i % 8): its L2 holds them for all.
constexpr int kStage = 128;

// Buffers: as many as one workgroup of 8 waves, or two of 4, have room for.
constexpr int buffers_of(int waves) { return waves == 8 ? 4 : 2; }
constexpr int many_lds(int waves) { return buffers_of(waves) * (kStage * 256 + kStage * 4) + waves * 512; }
template <int R, int WAVES, bool CAP>
__global__ __launch_bounds__(64 * WAVES, 2) void many_rows_kernel(PagedCache kv, TreeQueries tq, AttentionPlan plan,
                                                                  uint16_t* __restrict__ out, float* __restrict__ lse,
                                                                  float* __restrict__ part, int32_t* __restrict__ shares,
                                                                  uint32_t groups, uint32_t grid, uint32_t fill) {
    if (blockIdx.x >= grid) {
        fill_rows(tq, fill, out, lse, blockIdx.x - grid, gridDim.x - grid);
        return;
    }
    constexpr int kRuns = kStage / 8 / WAVES;  // of 8 rows of K, and of V, that a wave brings in
    constexpr int kBufs = buffers_of(WAVES);
    static_assert(kBufs * 8 * kRuns == 64, "a wave's block numbers of kBufs tiles are one load");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    uint32_t* present = reinterpret_cast<uint32_t*>(lds + kBufs * kStage * 256);  // [kBufs][kStage]
    uint32_t* pages = present + kBufs * kStage;                                   // [WAVES][2][64]
    const uint32_t lds0 = lds_address(lds);
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t hl = lane >> 5, n32 = lane & 31u;
    uint32_t id = blockIdx.x, rb = 0;
    if (plan.row_blocks > 1) {
        const uint32_t slot = id >> 3;
        rb = slot % plan.row_blocks;
        id = slot / plan.row_blocks * 8 + (id & 7u);
        if (id >= groups) return;
    }
    int32_t b, h, split, splits, share;
    if (plan.splits > 1) {
        const Shares r = shares_of<kStage>(tq, plan.groups, plan.split_tiles, (int32_t)id, lane);
        if (r.b < 0) return;
        b = r.b, h = r.h, split = r.split, splits = r.splits, share = r.tiles;
        // for the join: each sequence's first group and its splits
        if (rb == 0 && h == 0 && split == 0 && tid == 0) {
            shares[2 * b] = r.first;
            shares[2 * b + 1] = splits;
        }
    } else {
        b = id / tq.H, h = id % tq.H, split = 0, splits = 1, share = 1 << 30;
    }
    b = __builtin_amdgcn_readfirstlane(b);
    h = __builtin_amdgcn_readfirstlane(h);
    split = __builtin_amdgcn_readfirstlane(split);
    splits = __builtin_amdgcn_readfirstlane(splits);
    share = __builtin_amdgcn_readfirstlane(share);
    const Span s = span_of<kStage>(tq, b);
    const int32_t block0 = rb * WAVES * 32 * R;
    const int32_t first = split * share;
    if (block0 >= s.rows || first >= s.all_tiles) return;
    int32_t end = s.all_tiles - first < share ? s.all_tiles : first + share;
    const int32_t last = last_tile<kStage>(tq, s, block0 + WAVES * 32 * R - 1);
    if (end > last) end = last;
    const int32_t ctx_full = s.ctx / kStage;
    const int32_t row0 = block0 + (int32_t)wave * 32 * R;
    const bool active = row0 < s.rows;

    const uint16_t* head = kv.cache + (int64_t)h * kv.head_stride;
    const int32_t* table = kv.tables + (int64_t)b * kv.table_stride;
    const Factors f = factors<CAP>(tq);
    // Run i of the wave: 8 keys, a lane key lane / 8, the chunks that belong in place lane % 8 of its rows.
    int64_t off[kRuns];
    const uint32_t row8 = lane >> 3, c8 = lane & 7u;
    auto find = [&](int32_t t, int32_t stop) {
        if (t >= stop) return;
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            const uint32_t k = 8 * (kRuns * wave + i) + row8;
            off[i] = k < keys_from<kStage>(s, t) ? key_offset(kv, table, (uint32_t)t * kStage + k) : -1;
        }
    };
    // (a key that is not there is read from the cache's first cell, and masked)
    auto bring = [&](int buf, const int64_t (&off)[kRuns]) {
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            const uint32_t at = lds0 + buf * (kStage * 256) + (kRuns * wave + i) * 1024;
            const uint16_t* row = head + (off[i] >= 0 ? off[i] : 0);
            to_lds(row + 8 * (c8 ^ row8), at);
            to_lds(row + kHeadDim + 8 * (c8 ^ (row8 >> 1 & 1u) << 2), at + kStage * 128);
            if (c8 == 0) present[buf * kStage + 8 * (kRuns * wave + i) + row8] = off[i] >= 0;
        }
    };
    auto ballots = [&](int buf, uint64_t (&exists)[kStage / 64]) {
        bool all = true;
#pragma unroll
        for (int i = 0; i < kStage / 64; ++i) {
            exists[i] = __ballot(present[buf * kStage + 64 * i + lane] != 0u);
            all &= exists[i] == ~0ull;
        }
        return all;
    };
    // this lane's places in a stage
    const uint32_t k_at = n32 * 128, k_c = n32 & 7u, t16 = lane & 15u;
    const uint32_t v_at = kStage * 128 + (4 * hl + (t16 >> 2)) * 128 +
                          ((2 * (lane >> 4 & 1u) + (t16 >> 1 & 1u)) ^ (t16 >> 3) << 2) * 16 + (t16 & 1u) * 8;
    auto read_k = [&](Keys32& k, int buf, int sub) {
        const uint8_t* at = lds + buf * (kStage * 256) + sub * 4096 + k_at;
#pragma unroll
        for (int i = 0; i < 4; ++i) k.k[i] = load16(at + (((2 * i + hl) ^ k_c) << 4));
    };
    auto read_v = [&](Keys32& k, int buf, int sub) {
        const uint32_t at = buf * (kStage * 256) + sub * 4096;
        auto four = [&](uint32_t o) {
            typedef __attribute__((address_space(3))) i16x4 LdsFour;
            return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsFour*)(uintptr_t)(lds0 + o)));
        };
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const uint2 a = four(at + (v_at ^ c * 64) + ks * 2048), z = four(at + (v_at ^ c * 64) + ks * 2048 + 1024);
                k.v[c][ks] = U32x4{a.x, a.y, z.x, z.y};
            }
    };

    Rows32<R> w;
    int32_t node[R];  // of row l % 32 of each tile, -1 past the last row
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        const int32_t r = row0 + 32 * rt + (int32_t)n32;
        node[rt] = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) w.q[rt][i] = U32x4{0u, 0u, 0u, 0u};
        if (r < s.rows) {
            node[rt] = r / tq.G;
            const uint16_t* q = tq.q + (int64_t)(s.nodes.first + node[rt]) * tq.q_rs +
                                (int64_t)(h * tq.G + r - node[rt] * tq.G) * tq.q_hs + 8 * hl;
#pragma unroll
            for (int i = 0; i < 4; ++i) w.q[rt][i] = load16(q + 16 * i);
        }
        w.o[rt][0] = w.o[rt][1] = f32x16{0.f};
        w.base[rt] = kNone;
        w.c[rt] = f.c;
        w.l[rt] = 0.0f;
    }

    // The tiles that every row sees whole. One row tile's scores are on the way in the matrix cores while the
    // vector unit takes the other's exponentials (of one row tile: the next 32 keys' scores).
    constexpr int kSubs = kStage / 32;
    bool left_out = false;  // a tile of the context with a key that is not there
    const int32_t full_end = end < ctx_full ? end : ctx_full;
    if (first < full_end) {
        Keys32 k;
        f32x16 s0, s1;  // scores: of row tile 0 and 1 (of one row tile: of even and odd 32 keys)
        uint64_t exists[kStage / 64];
        // Block numbers go to LDS too, kBufs tiles of the wave's keys in one load and two such sets: a load to a register
        // would have the compiler wait for it, and with it for the tiles on the way.
        const int32_t all = full_end - first;
        uint32_t* own_pages = pages + wave * 128;
        auto find_pages = [&](int32_t set) {
            const int32_t t = first + set * kBufs + (int32_t)(lane / (8 * kRuns));
            const uint32_t key = (uint32_t)(t < full_end ? t : full_end - 1) * kStage + 8 * kRuns * wave + lane % (8 * kRuns);
            const uint32_t blk = block_of(key, kv);
            to_lds4(table + (blk < kv.table_width ? blk : kv.table_width - 1), lds_address(own_pages + (set & 1) * 64));
        };
        uint32_t page[kRuns];
        auto read_pages = [&](int32_t i) {
#pragma unroll
            for (int r = 0; r < kRuns; ++r) page[r] = own_pages[(i % (2 * kBufs)) * 8 * kRuns + 8 * r + row8];
        };
        auto bring_whole = [&](int32_t i) {
            int64_t offs[kRuns];
#pragma unroll
            for (int r = 0; r < kRuns; ++r) {
                offs[r] = key_offset(kv, (uint32_t)(first + i) * kStage + 8 * (kRuns * wave + r) + row8, page[r]);
            }
            bring(i % kBufs, offs);
        };
        // All but the loads of `later` tiles have landed; everybody's after the barrier.
        auto landed_but = [&](int32_t later) {
            if (later >= 3)
                wait_vmcnt<6 * kRuns>();
            else if (later == 2)
                wait_vmcnt<4 * kRuns>();
            else if (later == 1)
                wait_vmcnt<2 * kRuns>();
            else
                wait_vmcnt<0>();
            barrier();
        };
        find_pages(0);
        find_pages(1);
        wait_vmcnt<0>();
        for (int32_t i = 0; i < kBufs && i < all; ++i) {
            read_pages(i);
            bring_whole(i);
        }
        landed_but((all < kBufs ? all : kBufs) - 1);
        bool whole = ballots(0, exists), primed = false;
        for (int32_t i = 0; i < all; ++i) {
            const int buf = i % kBufs, next = (i + 1) % kBufs;
            const bool work = whole && active;
            read_pages(i + kBufs);
            if (work) {
                if (!primed) {
                    read_k(k, buf, 0);
                    scores32<R>(s0, w, 0, k);
                }
#pragma unroll
                for (int sub = 0; sub < kSubs; ++sub) {
                    read_v(k, buf, sub);
                    if constexpr (R == 2) {
                        scores32<R>(s1, w, 1, k);
                        add32<R, CAP, false>(w, 0, s0, k, f, 0u);
                        if (sub + 1 < kSubs) {
                            read_k(k, buf, sub + 1);
                            scores32<R>(s0, w, 0, k);
                            add32<R, CAP, false>(w, 1, s1, k, f, 0u);
                        }
                    } else if (sub + 1 < kSubs) {
                        read_k(k, buf, sub + 1);
                        scores32<R>(sub % 2 ? s0 : s1, w, 0, k);
                        add32<R, CAP, false>(w, 0, sub % 2 ? s1 : s0, k, f, 0u);
                    }
                }
            }
            // the wave has what it needs of this buffer
            const int32_t last_on_way = i + kBufs - 1 < all ? i + kBufs - 1 : all - 1;
            landed_but(last_on_way - (i + 1));
            if (i + kBufs < all) bring_whole(i + kBufs);
            if (buf == 0) find_pages(i / kBufs + 2);
            const bool next_whole = i + 1 < all && ballots(next, exists);
            primed = work && next_whole;
            if (primed) {
                read_k(k, next, 0);
                scores32<R>(s0, w, 0, k);
            }
            if (work) add32<R, CAP, false>(w, R - 1, s1, k, f, 0u);
            if (!whole) left_out = true;
            whole = next_whole;
        }
        landed();  // (nobody reads the buffers any more, and no block numbers are on the way)
    }
    // the others: the context's last, the nodes', those left out
    const int32_t rest = left_out || first > full_end ? first : full_end;
    if (rest < end) {
        find(rest, end);
        bring(0, off);
        find(rest + 1, end);
        for (int32_t t = rest; t < end; ++t) {
            const int buf = (t - rest) & 1;
            const bool has_nodes = (t + 1) * kStage > s.ctx;
            uint32_t words[R][kSubs];  // what the lane's rows see of the tile
#pragma unroll
            for (int rt = 0; rt < R; ++rt) seen_keys<kSubs>(words[rt], tq, s.nodes, s.ctx, node[rt], t * kStage);
            landed();
            if (t + 1 < end) bring(buf ^ 1, off);
            find(t + 2, end);
            uint64_t exists[kStage / 64];
            const bool whole = ballots(buf, exists);
            if (!active || (whole && t < ctx_full)) continue;
#pragma unroll 1
            for (int sub = 0; sub < kSubs; ++sub) {
                const uint32_t there = (uint32_t)((sub & 2 ? exists[1] : exists[0]) >> (32 * (sub & 1)));
                uint32_t word[R];
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    word[rt] = words[rt][0];
#pragma unroll
                    for (int i = 1; i < kSubs; ++i) words[rt][i - 1] = words[rt][i];
                }
                if (there == 0u) continue;
                Keys32 k;
                const uint32_t mine = bits_of_scores(there, hl);
                auto clear_absent = [&]() {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks) {
                            uint32_t* v = &k.v[c][ks].x;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t two = mine >> (8 * ks + 2 * j);
                                v[j] &= (two & 1u ? 0xFFFFu : 0u) | (two & 2u ? 0xFFFF0000u : 0u);
                            }
                        }
                };
                read_k(k, buf, sub);
                read_v(k, buf, sub);
                if (there != 0xFFFFFFFFu) clear_absent();
                bool odd = false;  // infinities and NaN in nodes' V: see add_odd
                if (has_nodes) {
                    u16x2 most{0, 0};
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        most = __builtin_elementwise_max(
                            most, __builtin_bit_cast(u16x2, (&k.v[i / 8][i / 4 % 2].x)[i % 4] & 0x7FFF7FFFu));
                    odd = __any(most.x >= 0x7F80 || most.y >= 0x7F80);
                    if (odd) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            uint32_t& v = (&k.v[i / 8][i / 4 % 2].x)[i % 4];
                            v = finite_pair(v);
                        }
                    }
                }
                uint32_t seen[R];
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    seen[rt] = bits_of_scores(there & word[rt], hl);
                    f32x16 sc;
                    scores32<R>(sc, w, rt, k);
                    add32<R, CAP, true>(w, rt, sc, k, f, seen[rt]);
                }
                if (!odd) continue;
                read_v(k, buf, sub);
                clear_absent();
#pragma unroll 1
                for (int kind = 0; kind < 3; ++kind) {
                    const float adds = kind == 0 ? __builtin_inff() : kind == 1 ? -__builtin_inff() : __builtin_nanf("");
                    const uint32_t which = kind == 0 ? 0x7F80u : kind == 1 ? 0xFF80u : 0u;
#pragma unroll
                    for (int rt = 0; rt < R; ++rt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            f32x16 met{0.f};
#pragma unroll
                            for (int ks = 0; ks < 2; ++ks) {
                                U32x4 ones, sees;
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    (&ones.x)[j] = ones_of_kind((&k.v[c][ks].x)[j], which);
                                    const uint32_t two = seen[rt] >> (8 * ks + 2 * j);
                                    (&sees.x)[j] = (two & 1u ? 0x3F80u : 0u) | (two & 2u ? 0x3F800000u : 0u);
                                }
                                met = mfma32(ones, sees, met);
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (met[i] > 0.0f) w.o[rt][c][i] += adds;
                        }
                }
            }
        }
    }
    if (!active) return;
    const int32_t heads = tq.H * tq.G;
    constexpr int kRows = WAVES * 32 * R;
    const int64_t part0 = ((int64_t)id * plan.row_blocks + rb) * kRows - block0;
    const Results to{out, lse, part, part + (int64_t)plan.groups * plan.row_blocks * kRows * kHeadDim, splits == 1};
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        const float l = w.l[rt] + lane_xor<32>(w.l[rt]);
        const float top = base_of<CAP>(w.base[rt], w.c[rt], f.c);
        if (node[rt] < 0) continue;
        const int32_t r = row0 + 32 * rt + (int32_t)n32;
        const int64_t at = splits > 1 ? part0 + r
                                      : (int64_t)(s.nodes.first + node[rt]) * heads + h * tq.G + r - node[rt] * tq.G;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                put_row4(to, at, 32 * c + 8 * i + 4 * (int32_t)hl, top, l,
                         f32x4{w.o[rt][c][4 * i], w.o[rt][c][4 * i + 1], w.o[rt][c][4 * i + 2], w.o[rt][c][4 * i + 3]});
    }
}

// The splits of a row joined: 16 lanes a row, 4 elements of d a lane, eight splits' loads on the way at a
// time. Bound by the latency of one row's loads.
__global__ __launch_bounds__(256) void tree_attention_join_kernel(TreeQueries tq, AttentionPlan plan,
                                                                  const float* __restrict__ part,
                                                                  const int32_t* __restrict__ shares,
                                                                  uint16_t* __restrict__ out, float* __restrict__ lse) {
    const int32_t heads = tq.H * tq.G;
    const int32_t row = blockIdx.x * 16 + (int32_t)(threadIdx.x >> 4), d = 4 * (int32_t)(threadIdx.x & 15u);
    const int32_t b = blockIdx.y;
    const Nodes nodes = nodes_of(tq, b);
    if (row >= nodes.count * heads) return;
    const int64_t at = (int64_t)nodes.first * heads + row;
    int64_t from, step;  // the first split's row of the partial sums, and the next one's distance
    const float* ml;
    int32_t splits;
    if (plan.many) {
        const int32_t rows = 16 * plan.q_tiles * plan.waves;
        const int32_t node = row / heads, hq = row - node * heads, h = hq / tq.G, r = node * tq.G + hq - h * tq.G;
        splits = shares[2 * b + 1];
        if (splits <= 1) return;  // written whole
        step = (int64_t)plan.row_blocks * rows;
        from = ((int64_t)(shares[2 * b] + h * splits) * plan.row_blocks + r / rows) * rows + r % rows;
        ml = part + (int64_t)plan.groups * step * kHeadDim;
    } else {
        const int32_t ctx = context_of(tq, b);
        const int32_t tiles = (ctx + nodes.count + kTile - 1) / kTile;
        splits = (tiles + plan.split_tiles - 1) / plan.split_tiles;
        if (splits > plan.splits) splits = plan.splits;
        step = (int64_t)tq.T * heads;
        from = at;
        ml = part + plan.splits * step * kHeadDim;
    }
    const float* pm = ml + from * 2;
    const float* po = part + from * kHeadDim + d;
    float base = -__builtin_inff(), l = 0.0f;  // the largest base so far
    f32x4 o{0.f, 0.f, 0.f, 0.f};
    constexpr int kAtOnce = 8;
    for (int32_t s0 = 0; s0 < splits; s0 += kAtOnce) {
        f32x4 p[kAtOnce];
        float2 ml[kAtOnce];
        float top = base;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t s = s0 + j < splits ? s0 + j : s0;
            p[j] = *reinterpret_cast<const f32x4*>(po + s * step * kHeadDim);
            ml[j] = *reinterpret_cast<const float2*>(pm + s * step * 2);
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
            const float f = exp2_hw(ml[j].x - ref);
            l = __builtin_fmaf(ml[j].y, f, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(p[j][i], f, o[i]);
        }
        base = top;
    }
    if (base == -__builtin_inff()) base = 0.0f;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint2 w;
    w.x = pack_bf16(o[0] * inv, o[1] * inv);
    w.y = pack_bf16(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(out + at * kHeadDim + d) = w;
    if (d == 0) lse[at] = l == 0.0f ? -__builtin_inff() : (base + log2_hw(l)) * kLn2;
}

template <int R, int WAVES, bool CAP, bool PAGE16>
int launch_few(const TreeAttentionArgs& a, hipStream_t stream) {
    constexpr int kLds = WAVES * 16 * R * (kPad + 2) * 4;
    static_assert(kLds <= 65536, "above, the limit would have to be raised");
    const uint32_t groups = (uint32_t)a.tq.B * a.tq.H * a.plan.splits;
    hipLaunchKernelGGL((few_rows_kernel<R, WAVES, CAP, PAGE16>), dim3(groups + fill_groups(a)), dim3(64 * WAVES), kLds, stream, a.kv,
                       a.tq, a.plan, a.out, a.lse, a.part, groups, a.fill);
    return 0;
}

template <int R, int WAVES>
int launch_few(const TreeAttentionArgs& a, hipStream_t stream) {
    // (32-bit offsets of a page's rows)
    const bool page16 = a.kv.block_size % 16 == 0 && a.kv.page_stride < (1 << 24);
    if (a.tq.softcap > 0.0f)
        return page16 ? launch_few<R, WAVES, true, true>(a, stream) : launch_few<R, WAVES, true, false>(a, stream);
    return page16 ? launch_few<R, WAVES, false, true>(a, stream) : launch_few<R, WAVES, false, false>(a, stream);
}

template <int R, int WAVES, bool CAP>
int launch_many(const TreeAttentionArgs& a, hipStream_t stream) {
    const uint32_t groups = a.plan.splits > 1 ? (uint32_t)a.plan.groups : (uint32_t)a.tq.B * a.tq.H;
    const uint32_t grid = a.plan.row_blocks > 1 ? (groups + 7) / 8 * 8 * a.plan.row_blocks : groups;
    auto kernel = many_rows_kernel<R, WAVES, CAP>;
    static std::atomic<int> done[64] = {};
    if (raise_lds_limit(reinterpret_cast<const void*>(kernel), many_lds(WAVES), done) != 0) return -1;
    hipLaunchKernelGGL(kernel, dim3(grid + fill_groups(a)), dim3(64 * WAVES), many_lds(WAVES), stream, a.kv, a.tq, a.plan, a.out, a.lse, a.part,
                       a.shares, groups, grid, a.fill);
    return 0;
}

}  // namespace

AttentionPlan plan_tree_attention(int32_t B, int32_t H, int32_t G, int32_t max_nodes, int64_t max_ctx, bool capped,
                                  int32_t num_cus) {
    AttentionPlan p{};
    const int64_t rows = (int64_t)max_nodes * G;
    // 64 sequences of 4096 keys and 8 heads: 32 rows 67 us as few, 64 rows 90 as many (135 in tiles of 64 rows as few).
    p.many = rows > 32;
    p.splits = 1;
    if (p.many) {
        // 128 rows a workgroup, two of them a CU; above, 256 and one, with more keys on the way (32768 keys of 4
        // sequences and 8 heads, 256 rows: 111 us against 188 with waves of 64 rows). Above 256 rows of capped scores,
        // whose exponentials leave the registers for it, 512 and waves of 64 rows (512 rows: 279 against 308 us;
        // uncapped 288 against 221).
        p.waves = rows > 128 ? 8 : 4;
        p.q_tiles = capped && rows > 256 ? 4 : 2;
        const int64_t block_rows = 16 * p.q_tiles * p.waves;
        p.row_blocks = (int32_t)((rows + block_rows - 1) / block_rows);
        const int64_t at_once = num_cus * (p.waves == 8 ? 1 : 2);
        const int64_t tiles = (max_ctx + max_nodes + kStage - 1) / kStage;
        p.split_tiles = 2;
        p.groups = (int32_t)(at_once / p.row_blocks);
        // split when the chip has room for twice the workgroups, by what the lengths turn out to be
        if (2 * (int64_t)B * H <= p.groups && tiles > p.split_tiles) p.splits = 2;
        return p;
    }
    p.q_tiles = rows <= 16 ? 1 : 2;
    p.waves = 4;
    p.row_blocks = 1;
    const int64_t tiles = (max_ctx + max_nodes + kTile - 1) / kTile;
    const int64_t base = (int64_t)B * H;
    if (p.q_tiles == 1 && tiles <= 64 && base <= num_cus) {
        // Short and few: 8 waves, 8 tiles each at most, and no second launch (8 heads: 1000 keys 10.5 us a launch, 16
        // waves of half the registers 11.7; a call at 2000 keys 18 us, split in two launches 21; at 4000 split 21, one 27).
        p.waves = 8;
        p.split_tiles = (int32_t)tiles;
        return p;
    }
    // Splits until there are two workgroups per CU, each of at least 4 tiles a wave.
    int64_t splits = (2 * num_cus + base - 1) / base;
    const int64_t most = tiles / (4 * p.waves);
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    p.split_tiles = (int32_t)((tiles + splits - 1) / splits);
    p.splits = (int32_t)((tiles + p.split_tiles - 1) / p.split_tiles);
    return p;
}

int64_t tree_attention_workspace(const AttentionPlan& p, int64_t T, int64_t heads, int32_t B) {
    if (p.splits == 1) return 0;
    const int64_t rows = p.many ? (int64_t)p.groups * p.row_blocks * 16 * p.q_tiles * p.waves : p.splits * T * heads;
    return rows * (kHeadDim + 2) * 4 + (p.many ? (int64_t)B * 2 * 4 : 0);
}

int launch_tree_attention(const TreeAttentionArgs& a, hipStream_t stream) {
    int rc;
    const bool capped = a.tq.softcap > 0.0f;
    if (a.tq.B == 0) {
        hipLaunchKernelGGL(fill_rows_kernel, dim3(fill_groups(a)), dim3(256), 0, stream, a.tq, a.fill, a.out, a.lse);
        return hipGetLastError() == hipSuccess ? 0 : -1;
    }
    if (a.plan.many)
        rc = a.plan.q_tiles == 4 ? launch_many<2, 8, true>(a, stream)
             : a.plan.waves == 8 ? (capped ? launch_many<1, 8, true>(a, stream) : launch_many<1, 8, false>(a, stream))
             : capped            ? launch_many<1, 4, true>(a, stream)
                                 : launch_many<1, 4, false>(a, stream);
    else if (a.plan.waves == 8)
        rc = launch_few<1, 8>(a, stream);
    else
        rc = a.plan.q_tiles == 1 ? launch_few<1, 4>(a, stream) : launch_few<2, 4>(a, stream);
    if (rc) return rc;
    if (a.plan.splits > 1) {
        const dim3 grid((uint32_t)(((int64_t)a.tq.max_nodes * a.tq.H * a.tq.G + 15) / 16), (uint32_t)a.tq.B);
        hipLaunchKernelGGL(tree_attention_join_kernel, grid, dim3(256), 0, stream, a.tq, a.plan, a.part, a.shares, a.out,
                           a.lse);
    }
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
