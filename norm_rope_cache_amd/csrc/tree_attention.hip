// Attention of drafted tokens over the paged cache.
//
// s_ij = scale q_i . k_j (capped: cap tanh(s / cap)), p = softmax over the
// keys that node i sees, out_i = sum_j p_ij v_j, lse_i = log sum_j e^(s_ij).
// A sequence's keys are its context, which every node sees, and its nodes,
// seen as the tree mask says.
//
// One pass over the keys with a running maximum m and sum l per query row.
// A tile is 32 keys by 16 query rows (rows = nodes x the query heads of one KV
// head, so every cached byte is fetched once for all of them):
//   S^T = K Q^T   4 v_mfma_f32_16x16x32_bf16; A is K as it lies (lane: key
//                 l % 16, 8 elements of d), so K goes from memory to the matrix
//                 core without LDS. A lane then holds, for query row l % 16, the
//                 keys 4 (l / 16) + r of both halves of the tile.
//   O^T += V^T P^T  4 more. P^T's lane needs 8 keys of query row l % 16: the
//                 ones it holds, when slot 8 g + 4 t + r of the sum stands for
//                 key 16 t + 4 g + r. V's lane loads those same 8 keys, 4 elements of
//                 d each (8 bytes), and 16 byte permutes turn them into the 4
//                 operands (operand c: d = 4 (l % 16) + c).
// The statistics of a row and its column of O^T thus live in the lanes that
// hold its scores. P is rounded to bf16 for the second product (relative 2^-9
// each, independent between keys, so the error of the sum stays near the bf16
// output's own rounding); m, l, O and the scores are FP32.
//
// m moves only when a score passes it by 2^8 (the lanes vote): between, p and
// l and O grow by up to that factor, which FP32 and bf16 hold at full precision,
// and no lane waits for another lane's maximum.
#include "cache_ops.h"
#include "kernels.h"
#include "paged.h"

namespace nrc {
namespace {

constexpr int kTile = 32;
constexpr int kPad = 68;  // floats to a row of O in LDS (64 and 4 against bank conflicts)

// The 32 keys of a tile in registers: K as S's A operand (tile half t, half h
// of d), V's 8 keys with 4 elements of d.
struct Keys {
    U32x4 k[2][2];
    uint2 v[8];
};

__device__ __forceinline__ float group_max(float x) {
    x = __builtin_fmaxf(x, lane_xor<16>(x));
    return __builtin_fmaxf(x, lane_xor<32>(x));
}
__device__ __forceinline__ float group_sum(float x) {
    x = x + lane_xor<16>(x);
    return x + lane_xor<32>(x);
}

// V's rows as the A operand of element c of every lane's four: the 8 keys' c-th.
__device__ __forceinline__ U32x4 v_operand(const Keys& kv, int c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = c < 2 ? kv.v[2 * i].x : kv.v[2 * i].y;
        const uint32_t b = c < 2 ? kv.v[2 * i + 1].x : kv.v[2 * i + 1].y;
        w[i] = __builtin_amdgcn_perm(b, a, c % 2 ? 0x07060302u : 0x05040100u);
    }
    return U32x4{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ bool inf_or_nan_pair(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// What a wave carries for R query tiles of 16 rows.
template <int R>
struct Rows {
    U32x4 q[R][2];   // S's B operand: row l % 16, halves of d
    f32x4 o[R][4];   // O^T: row l % 16, d = 4 (4 (l / 16) + r) + c at [c][r]
    float m[R];      // the running maximum, raw scores (-inf: none yet)
    float base[R];   // subtracted from the scores in base 2: m's, or 0 without one
    float l[R];      // this lane's share of the sum
};

template <bool CAP>
__device__ __forceinline__ float in_base2(float raw, float c, float capped) {
    if constexpr (CAP) return __builtin_fmaf(rcp_hw(exp2_hw(raw * c) + 1.0f), -2.0f * capped, capped);
    return raw * c;
}

// One tile. c: raw scores to base 2 (scale log2 e), or with CAP to the
// exponent of tanh (2 scale log2 e / cap), capped then being cap log2 e.
// MASKED: seen[rq] has this lane's rows' bits of the tile's keys.
template <int R, bool CAP, bool MASKED>
__device__ __forceinline__ void tile(Rows<R>& w, const Keys& kv, float c, float capped, float slack,
                                     const uint32_t (&seen)[R], uint32_t lane) {
    const uint32_t g = lane >> 4;
    U32x4 va[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) va[i] = v_operand(kv, i);
#pragma unroll
    for (int rq = 0; rq < R; ++rq) {
        f32x4 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = mfma16(kv.k[t][0], w.q[rq][0], f32x4{0.f, 0.f, 0.f, 0.f});
            s[t] = mfma16(kv.k[t][1], w.q[rq][1], s[t]);
        }
        if constexpr (MASKED) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!(seen[rq] >> (16 * t + 4 * g + r) & 1u)) s[t][r] = -__builtin_inff();
        }
        float top = __builtin_fmaxf(__builtin_fmaxf(__builtin_fmaxf(s[0][0], s[0][1]), __builtin_fmaxf(s[0][2], s[0][3])),
                                    __builtin_fmaxf(__builtin_fmaxf(s[1][0], s[1][1]), __builtin_fmaxf(s[1][2], s[1][3])));
        // (slack: 8 in raw scores; the cap only brings scores nearer to each other)
        if (__any(top > w.m[rq] + slack)) {
            const float m = __builtin_fmaxf(w.m[rq], group_max(top));
            const float base = m == -__builtin_inff() ? 0.0f : in_base2<CAP>(m, c, capped);
            // -inf before: no key yet, l and O are 0
            const float shrink = w.m[rq] == -__builtin_inff() ? 1.0f : exp2_hw(w.base[rq] - base);
            w.l[rq] *= shrink;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) w.o[rq][i][r] *= shrink;
            w.m[rq] = m;
            w.base[rq] = base;
        }
        float p[8];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float e;
                if constexpr (CAP) {
                    e = __builtin_fmaf(rcp_hw(exp2_hw(s[t][r] * c) + 1.0f), -2.0f * capped, capped - w.base[rq]);
                    if (MASKED && !(seen[rq] >> (16 * t + 4 * g + r) & 1u)) e = -__builtin_inff();
                } else {
                    e = __builtin_fmaf(s[t][r], c, -w.base[rq]);
                }
                p[4 * t + r] = exp2_hw(e);
            }
        w.l[rq] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        const U32x4 pb{pack_bf16_pair_hw(p[0], p[1]), pack_bf16_pair_hw(p[2], p[3]), pack_bf16_pair_hw(p[4], p[5]),
                       pack_bf16_pair_hw(p[6], p[7])};
#pragma unroll
        for (int i = 0; i < 4; ++i) w.o[rq][i] = mfma16(va[i], pb, w.o[rq][i]);
    }
}

// K and V of a tile from its keys' addresses: lane l < 32 holds the offset of
// key l (elements, head 0; < 0: no such key). K of an absent key is read as 0 and
// masked by the caller, V as 0.
__device__ __forceinline__ void load_keys(Keys& kv, const uint16_t* head, int64_t off, uint32_t lane) {
    const uint32_t g = lane >> 4, n = lane & 15u;
    auto of = [&](uint32_t key) {
        const int lo = __builtin_amdgcn_ds_bpermute((int)(key << 2), (int)(uint32_t)off);
        const int hi = __builtin_amdgcn_ds_bpermute((int)(key << 2), (int)(uint32_t)((uint64_t)off >> 32));
        return (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
    };
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int64_t o = of(16 * t + n);
        kv.k[t][0] = kv.k[t][1] = U32x4{0u, 0u, 0u, 0u};
        if (o >= 0) {
            kv.k[t][0] = load16(head + o + 8 * g);
            kv.k[t][1] = load16(head + o + 32 + 8 * g);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t ov = of(16 * t + 4 * g + r);
            kv.v[4 * t + r] = uint2{0u, 0u};
            if (ov >= 0) kv.v[4 * t + r] = *reinterpret_cast<const uint2*>(head + ov + kHeadDim + 4 * n);
        }
    }
}

// A tile of which some rows do not see some keys. Infinities and NaN in V
// reach only the rows that see their key: they leave V for the products
// (0 times them would be NaN in every row), and a product of "sees the key" with
// "is +inf / -inf / NaN there" tells each row which of them it meets.
template <int R, bool CAP>
__device__ __forceinline__ void masked_tile(Rows<R>& w, Keys& kv, float c, float capped, float slack,
                                            const uint32_t (&seen)[R], uint32_t lane) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) odd = odd || inf_or_nan_pair(kv.v[i].x) || inf_or_nan_pair(kv.v[i].y);
    if (!__any(odd)) {
        tile<R, CAP, true>(w, kv, c, capped, slack, seen, lane);
        return;
    }
    Keys kinds[3];  // 1.0 where V is +inf, -inf, NaN
    auto sort_out = [&](uint32_t& v, uint32_t& p, uint32_t& n, uint32_t& q) {
        p = n = q = 0u;
#pragma unroll
        for (int s = 0; s < 32; s += 16) {
            const uint32_t e = v >> s & 0xFFFFu;
            if ((e & 0x7F80u) != 0x7F80u) continue;
            if (e == 0x7F80u) p |= 0x3F80u << s;
            else if (e == 0xFF80u) n |= 0x3F80u << s;
            else q |= 0x3F80u << s;
            v &= ~(0xFFFFu << s);
        }
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sort_out(kv.v[i].x, kinds[0].v[i].x, kinds[1].v[i].x, kinds[2].v[i].x);
        sort_out(kv.v[i].y, kinds[0].v[i].y, kinds[1].v[i].y, kinds[2].v[i].y);
    }
    tile<R, CAP, true>(w, kv, c, capped, slack, seen, lane);
#pragma unroll
    for (int rq = 0; rq < R; ++rq) {
        uint32_t sees[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t bit = 16 * (i / 2) + 4 * (lane >> 4) + 2 * (i % 2);
            sees[i] = (seen[rq] >> bit & 1u ? 0x3F80u : 0u) | (seen[rq] >> (bit + 1) & 1u ? 0x3F800000u : 0u);
        }
        const U32x4 sb{sees[0], sees[1], sees[2], sees[3]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 met[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) met[k] = mfma16(v_operand(kinds[k], i), sb, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (met[0][r] > 0.0f) w.o[rq][i][r] += __builtin_inff();
                if (met[1][r] > 0.0f) w.o[rq][i][r] -= __builtin_inff();
                if (met[2][r] > 0.0f) w.o[rq][i][r] = __builtin_nanf("");
            }
        }
    }
}

// Grid: one workgroup per (sequence, KV head, split, block of 16 R query
// rows); its WAVES waves hold the same rows and take the split's tiles in turn,
// and join their sums in LDS. The row blocks of one split, which read the same
// keys, run on one XCD next to each other (workgroup i runs on XCD i % 8), so
// its L2 holds those keys for all of them.
template <int R, int WAVES, bool CAP>
__global__ __launch_bounds__(64 * WAVES) void tree_attention_kernel(PagedCache kv, TreeQueries tq, AttentionPlan plan,
                                                                    uint16_t* __restrict__ out,
                                                                    float* __restrict__ lse, float* __restrict__ part,
                                                                    uint32_t groups) {
    extern __shared__ float smem[];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t g = lane >> 4, n16 = lane & 15u;
    uint32_t id = blockIdx.x, rb = 0;
    if (plan.row_blocks > 1) {
        const uint32_t slot = id >> 3;
        rb = slot % plan.row_blocks;
        id = slot / plan.row_blocks * 8 + (id & 7u);
        if (id >= groups) return;
    }
    const int32_t split = id % plan.splits;
    const uint32_t bh = id / plan.splits;
    const int32_t h = bh % tq.H, b = bh / tq.H;
    const Nodes nodes = nodes_of(tq, b);
    const int32_t ctx = context_of(tq, b);
    const int32_t rows = nodes.count * tq.G, row0 = rb * 16 * R;
    if (row0 >= rows) return;
    const int32_t heads = tq.H * tq.G;

    // The tiles: the context's, then the nodes' (a chain: up to the last of this block's).
    const int32_t ctx_tiles = (ctx + kTile - 1) / kTile, ctx_full = ctx / kTile;
    const int32_t all_tiles = ctx_tiles + (nodes.count + kTile - 1) / kTile;
    const int32_t first = split * plan.split_tiles;
    if (first >= all_tiles) return;  // nor does the join look at this split
    int32_t end = first + plan.split_tiles < all_tiles ? first + plan.split_tiles : all_tiles;
    int32_t last_row = row0 + 16 * R - 1;
    if (last_row >= rows) last_row = rows - 1;
    if (!tq.mask) {
        const int32_t need = ctx_tiles + last_row / tq.G / kTile + 1;
        if (end > need) end = need;
    }

    Rows<R> w;
    int32_t node[R];  // the lane's rows' nodes, -1 past the last row
#pragma unroll
    for (int rq = 0; rq < R; ++rq) {
        const int32_t r = row0 + 16 * rq + n16;
        node[rq] = -1;
        w.q[rq][0] = w.q[rq][1] = U32x4{0u, 0u, 0u, 0u};
        if (r < rows) {
            node[rq] = r / tq.G;
            const uint16_t* q = tq.q + (int64_t)(nodes.first + node[rq]) * tq.q_rs +
                                (int64_t)(h * tq.G + r - node[rq] * tq.G) * tq.q_hs + 8 * g;
            w.q[rq][0] = load16(q);
            w.q[rq][1] = load16(q + 32);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w.o[rq][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        w.m[rq] = -__builtin_inff();
        w.base[rq] = 0.0f;
        w.l[rq] = 0.0f;
    }
    const float c = CAP ? 2.0f * kLog2E * tq.scale / tq.softcap : kLog2E * tq.scale;
    const float capped = CAP ? tq.softcap * kLog2E : 0.0f;
    const float slack = 8.0f / (kLog2E * tq.scale);
    const uint16_t* head = kv.cache + (int64_t)h * kv.head_stride;
    const int32_t* table = kv.tables + (int64_t)b * kv.table_stride;

    for (int32_t t = first + wave; t < end; t += WAVES) {
        const int32_t in_tree = t - ctx_tiles;  // >= 0: a tile of nodes
        const uint32_t key0 = in_tree < 0 ? (uint32_t)t * kTile : (uint32_t)(ctx + in_tree * kTile);
        const uint32_t there = in_tree < 0 ? (uint32_t)(ctx - t * kTile) : (uint32_t)(nodes.count - in_tree * kTile);
        int64_t off = -1;
        if (lane < kTile && lane < there) off = key_offset(kv, table, key0 + lane);
        const uint32_t exists = (uint32_t)__ballot(off >= 0);
        Keys keys;
        load_keys(keys, head, off, lane);
        uint32_t seen[R];
        if (exists == 0xFFFFFFFFu && t < ctx_full) {
            tile<R, CAP, false>(w, keys, c, capped, slack, seen, lane);
        } else {
#pragma unroll
            for (int rq = 0; rq < R; ++rq) {
                seen[rq] = exists;
                if (in_tree >= 0)
                    seen[rq] &= node[rq] < 0 ? 0u
                                             : seen_word(tq, nodes.first + node[rq], node[rq], nodes.count, in_tree);
            }
            masked_tile<R, CAP>(w, keys, c, capped, slack, seen, lane);
        }
    }

    // Join the waves: each leaves m's base, l and O of its rows in LDS.
    float* so = smem;                               // [WAVES][16 R][kPad]
    float* sm = smem + WAVES * 16 * R * kPad;       // [WAVES][16 R]
    float* sl = sm + WAVES * 16 * R;                // [WAVES][16 R]
#pragma unroll
    for (int rq = 0; rq < R; ++rq) {
        const float l = group_sum(w.l[rq]);
        const uint32_t row = wave * 16 * R + 16 * rq + n16;
        if (g == 0) {
            sm[row] = w.m[rq] == -__builtin_inff() ? -__builtin_inff() : w.base[rq];
            sl[row] = l;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) so[row * kPad + 16 * g + 4 * r + i] = w.o[rq][i][r];
    }
    __syncthreads();
    constexpr int kThreads = 64 * WAVES;
    for (int32_t e = threadIdx.x; e < 16 * R * 16; e += kThreads) {
        const int32_t lr = e >> 4, d = (e & 15) * 4;
        const int32_t r = row0 + lr;
        if (r >= rows) continue;
        float top = -__builtin_inff();
#pragma unroll
        for (int k = 0; k < WAVES; ++k) top = __builtin_fmaxf(top, sm[k * 16 * R + lr]);
        const float base = top == -__builtin_inff() ? 0.0f : top;
        float l = 0.0f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
            const float f = exp2_hw(sm[k * 16 * R + lr] - base);
            l = __builtin_fmaf(sl[k * 16 * R + lr], f, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(so[(k * 16 * R + lr) * kPad + d + i], f, o[i]);
        }
        const int32_t node_r = r / tq.G;
        const int64_t at = (int64_t)(nodes.first + node_r) * heads + h * tq.G + (r - node_r * tq.G);
        if (plan.splits > 1) {
            const int64_t rows_all = (int64_t)tq.T * heads;
            float* po = part + ((int64_t)split * rows_all + at) * kHeadDim + d;
            *reinterpret_cast<f32x4*>(po) = f32x4{o[0], o[1], o[2], o[3]};
            if (d == 0) {
                float* pm = part + (int64_t)plan.splits * rows_all * kHeadDim + ((int64_t)split * rows_all + at) * 2;
                pm[0] = top;
                pm[1] = l;
            }
        } else {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint32_t* po = reinterpret_cast<uint32_t*>(out + at * kHeadDim + d);
            po[0] = pack_bf16(o[0] * inv, o[1] * inv);
            po[1] = pack_bf16(o[2] * inv, o[3] * inv);
            if (d == 0) lse[at] = l == 0.0f ? -__builtin_inff() : (base + log2_hw(l)) * kLn2;
        }
    }
}

// The splits of a row joined, one wave per row, one element of d per lane.
__global__ __launch_bounds__(256) void tree_attention_join_kernel(TreeQueries tq, AttentionPlan plan,
                                                                  const float* __restrict__ part,
                                                                  uint16_t* __restrict__ out, float* __restrict__ lse) {
    const uint32_t lane = threadIdx.x & 63u;
    const int32_t heads = tq.H * tq.G;
    const int32_t hq = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int32_t i = blockIdx.y, b = blockIdx.z;
    const Nodes nodes = nodes_of(tq, b);
    if (i >= nodes.count || hq >= heads) return;
    const int32_t ctx = context_of(tq, b);
    const int32_t tiles = (ctx + kTile - 1) / kTile + (nodes.count + kTile - 1) / kTile;
    int32_t splits = (tiles + plan.split_tiles - 1) / plan.split_tiles;
    if (splits > plan.splits) splits = plan.splits;
    const int64_t rows_all = (int64_t)tq.T * heads;
    const int64_t at = (int64_t)(nodes.first + i) * heads + hq;
    const float* pm = part + (int64_t)plan.splits * rows_all * kHeadDim + at * 2;
    float top = -__builtin_inff();
    for (int32_t s = 0; s < splits; ++s) top = __builtin_fmaxf(top, pm[(int64_t)s * rows_all * 2]);
    const float base = top == -__builtin_inff() ? 0.0f : top;
    float l = 0.0f, o = 0.0f;
    for (int32_t s = 0; s < splits; ++s) {
        const float f = exp2_hw(pm[(int64_t)s * rows_all * 2] - base);
        l = __builtin_fmaf(pm[(int64_t)s * rows_all * 2 + 1], f, l);
        o = __builtin_fmaf(part[((int64_t)s * rows_all + at) * kHeadDim + lane], f, o);
    }
    out[at * kHeadDim + lane] = (uint16_t)to_bf16(l == 0.0f ? 0.0f : o / l);
    if (lane == 0) lse[at] = l == 0.0f ? -__builtin_inff() : (base + log2_hw(l)) * kLn2;
}

template <int R, int WAVES, bool CAP>
int launch(const TreeAttentionArgs& a, hipStream_t stream) {
    constexpr int kLds = WAVES * 16 * R * (kPad + 2) * 4;
    static std::atomic<int> done[64] = {};
    auto kernel = tree_attention_kernel<R, WAVES, CAP>;
    if (kLds > 65536 && raise_lds_limit(reinterpret_cast<const void*>(kernel), kLds, done) != 0) return -1;
    const uint32_t groups = (uint32_t)a.tq.B * a.tq.H * a.plan.splits;
    const uint32_t grid = a.plan.row_blocks > 1 ? (groups + 7) / 8 * 8 * a.plan.row_blocks : groups;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * WAVES), kLds, stream, a.kv, a.tq, a.plan, a.out, a.lse, a.part,
                       groups);
    return 0;
}

template <int R, int WAVES>
int launch_cap(const TreeAttentionArgs& a, hipStream_t stream) {
    return a.tq.softcap > 0.0f ? launch<R, WAVES, true>(a, stream) : launch<R, WAVES, false>(a, stream);
}

}  // namespace

AttentionPlan plan_tree_attention(int32_t B, int32_t H, int32_t G, int32_t max_nodes, int64_t max_ctx,
                                  int32_t num_cus) {
    AttentionPlan p{};
    const int64_t rows = (int64_t)max_nodes * G;
    p.q_tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    p.waves = 4;
    p.row_blocks = (int32_t)((rows + 16 * p.q_tiles - 1) / (16 * p.q_tiles));
    const int64_t tiles = (max_ctx + kTile - 1) / kTile + (max_nodes + kTile - 1) / kTile;
    // Splits until there are two workgroups per CU, each of at least 4 tiles a wave.
    const int64_t base = (int64_t)B * H * p.row_blocks;
    int64_t splits = (2 * num_cus + base - 1) / base;
    const int64_t most = tiles / (4 * p.waves);
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    p.split_tiles = (int32_t)((tiles + splits - 1) / splits);
    p.splits = (int32_t)((tiles + p.split_tiles - 1) / p.split_tiles);
    return p;
}

int launch_tree_attention(const TreeAttentionArgs& a, hipStream_t stream) {
    int rc;
    if (a.plan.q_tiles == 1)
        rc = launch_cap<1, 4>(a, stream);
    else if (a.plan.q_tiles == 2)
        rc = launch_cap<2, 4>(a, stream);
    else
        rc = launch_cap<4, 4>(a, stream);
    if (rc) return rc;
    if (a.plan.splits > 1) {
        const dim3 grid((uint32_t)(a.tq.H * a.tq.G + 3) / 4, (uint32_t)a.tq.max_nodes, (uint32_t)a.tq.B);
        hipLaunchKernelGGL(tree_attention_join_kernel, grid, dim3(256), 0, stream, a.tq, a.plan, a.part, a.out, a.lse);
    }
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
