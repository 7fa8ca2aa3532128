// What the attention kernels over a paged cache share: the running softmax of a tile
// of keys against 16 or 32 rows, infinities and NaN in V, the rows that a
// workgroup works on, where results go.
#pragma once

#include "../../include/nrc.h"
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
    float base[R];   // subtracted from the scores in base 2; kNone: no key yet
    float c[R];      // raw scores to base 2, see rebase
    float l[R];      // this lane's share of the sum
};

template <bool CAP>
__device__ __forceinline__ float in_base2(float raw, float c, float capped) {
    if constexpr (CAP) return __builtin_fmaf(rcp_hw(exp2_hw(raw * c) + 1.0f), -2.0f * capped, capped);
    return raw * c;
}

// Weights are taken against base as it stands; where a lane's sum passes kMost (or is NaN: the lanes vote), base moves
// to the row's largest score of the tile, and they are taken again. Under kNone any score's weight is +inf, that of
// -inf 0, so a row's first key moves it.
constexpr float kNone = -3.402823466e38f, kMost = 256.0f;

// Row's base moved up to its largest score `top`, if that is above it; what l and O shrink by.
// Past 2^30 the rounding of top c alone would overflow the exponential (2^6 and more), while scores that differ at all
// are 2^7 apart and more: there c's power of two takes its place, with which the largest score meets base exactly.
template <bool CAP>
__device__ __forceinline__ float rebase(float top, float& base, float& c, float whole_c, float capped) {
    const float at = CAP ? in_base2<CAP>(top, whole_c, capped) : top * c;
    if (top == -__builtin_inff() || !(at > base)) return 1.0f;
    const float shrink = exp2_hw(base - at);
    if constexpr (!CAP) {
        const float power = __uint_as_float(__float_as_uint(whole_c) & 0x7F800000u);
        c = __builtin_fabsf(top * whole_c) > 0x1p30f ? power : whole_c;
    }
    base = CAP ? at : top * c;
    return shrink;
}

// Of a row, for the join and lse: its base in base 2, -inf without a key.
template <bool CAP>
__device__ __forceinline__ float base_of(float base, float c, float whole_c) {
    return base == kNone ? -__builtin_inff() : CAP || c == whole_c ? base : base * (whole_c / c);
}

template <int R, bool CAP>
__device__ __forceinline__ void raise(Rows<R>& w, int rq, float top, float c, float capped) {
    const float shrink = rebase<CAP>(group_max(top), w.base[rq], w.c[rq], c, capped);
    w.l[rq] *= shrink;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) w.o[rq][i][r] *= shrink;
}

__device__ __forceinline__ float max8(const f32x4 (&s)[2]) {
    const float a = __builtin_fmaxf(__builtin_fmaxf(s[0][0], s[0][1]), s[0][2]);
    const float b = __builtin_fmaxf(__builtin_fmaxf(s[0][3], s[1][0]), s[1][1]);
    return __builtin_fmaxf(__builtin_fmaxf(__builtin_fmaxf(a, b), s[1][2]), s[1][3]);
}

// The weights of one query tile as the second product's operand; their sum. The operand is bf16, as V is: each weight is off by
// 2^-8 of itself at most, independently, and outputs by 0.0022 of their norm where FP32 weights would leave 0.0017 (the
// rounding of the outputs themselves). The sum is of the unrounded ones.
template <bool CAP>
__device__ __forceinline__ float open_weights(const f32x4 (&s)[2], float base, float c, float capped, U32x4& pb) {
    const float from = CAP ? capped - base : -base;
    float p[8];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            p[4 * t + r] = exp2_hw(CAP ? __builtin_fmaf(rcp_hw(exp2_hw(s[t][r] * c) + 1.0f), -2.0f * capped, from)
                                       : __builtin_fmaf(s[t][r], c, from));
    pb = U32x4{pack_bf16_pair_hw(p[0], p[1]), pack_bf16_pair_hw(p[2], p[3]), pack_bf16_pair_hw(p[4], p[5]),
               pack_bf16_pair_hw(p[6], p[7])};
    return ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
}

// A tile whose keys every row sees, two query tiles side by side: the products'
// latencies and the exponentials of one hide behind the other's, and their
// scores leave room in the registers.
template <int R, bool CAP>
__device__ __forceinline__ void open_tile(Rows<R>& w, const Keys& kv, float c, float capped) {
    constexpr int P = R < 2 ? 1 : 2;
#pragma unroll
    for (int r0 = 0; r0 < R; r0 += P) {
        f32x4 s[P][2];
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
            for (int t = 0; t < 2; ++t) s[j][t] = mfma16(kv.k[t][0], w.q[r0 + j][0], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
            for (int t = 0; t < 2; ++t) s[j][t] = mfma16(kv.k[t][1], w.q[r0 + j][1], s[j][t]);
        U32x4 pb[P];
        float sum[P];
        bool up = false;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            sum[j] = open_weights<CAP>(s[j], w.base[r0 + j], CAP ? c : w.c[r0 + j], capped, pb[j]);
            up = up || !(sum[j] <= kMost);
        }
        if (__any(up)) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                raise<R, CAP>(w, r0 + j, max8(s[j]), c, capped);
                sum[j] = open_weights<CAP>(s[j], w.base[r0 + j], CAP ? c : w.c[r0 + j], capped, pb[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < P; ++j) w.l[r0 + j] += sum[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const U32x4 va = v_operand(kv, i);
#pragma unroll
            for (int j = 0; j < P; ++j) w.o[r0 + j][i] = mfma16(va, pb[j], w.o[r0 + j][i]);
        }
    }
}

// One tile of which some rows may not see some keys. c: raw scores to base 2 (scale log2 e), or with CAP to the
// exponent of tanh (2 scale log2 e / cap), capped then being cap log2 e.
// seen[rq]: this lane's rows' bits of the tile's keys.
template <int R, bool CAP>
__device__ __forceinline__ void masked_tile(Rows<R>& w, const Keys& kv, float c, float capped,
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
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (!(seen[rq] >> (16 * t + 4 * g + r) & 1u)) s[t][r] = -__builtin_inff();
        U32x4 pb;
        auto weights = [&]() {
            float p[8];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float e;
                    if constexpr (CAP) {
                        e = __builtin_fmaf(rcp_hw(exp2_hw(s[t][r] * c) + 1.0f), -2.0f * capped, capped - w.base[rq]);
                        if (!(seen[rq] >> (16 * t + 4 * g + r) & 1u)) e = -__builtin_inff();
                    } else {
                        e = __builtin_fmaf(s[t][r], w.c[rq], -w.base[rq]);
                    }
                    p[4 * t + r] = exp2_hw(e);
                }
            pb = U32x4{pack_bf16_pair_hw(p[0], p[1]), pack_bf16_pair_hw(p[2], p[3]), pack_bf16_pair_hw(p[4], p[5]),
                       pack_bf16_pair_hw(p[6], p[7])};
            return ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        };
        float sum = weights();
        if (__any(!(sum <= kMost))) {
            raise<R, CAP>(w, rq, max8(s), c, capped);
            sum = weights();
        }
        w.l[rq] += sum;
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

// Infinities and NaN in the V of nodes, which not every row sees: they leave V
// for the products (0 times them would be NaN in every row), and afterwards a
// product of "sees the key" with "is +inf (or -inf, or NaN) there" tells each row
// which of them it meets.
__device__ __forceinline__ bool any_odd(const Keys& kv) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) odd = odd || inf_or_nan_pair(kv.v[i].x) || inf_or_nan_pair(kv.v[i].y);
    return __any(odd);
}
__device__ __forceinline__ uint32_t finite_pair(uint32_t v) {
    if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
    return (v & 0x7F800000u) == 0x7F800000u ? v & 0xFFFFu : v;
}
__device__ __forceinline__ void drop_odd(Keys& kv) {
#pragma unroll
    for (int i = 0; i < 8; ++i) kv.v[i] = uint2{finite_pair(kv.v[i].x), finite_pair(kv.v[i].y)};
}
// The elements of one kind as 1.0: which is 0x7F80 (+inf), 0xFF80 (-inf) or 0 (NaN).
__device__ __forceinline__ uint32_t ones_of_kind(uint32_t v, uint32_t which) {
    uint32_t w = 0u;
#pragma unroll
    for (int s = 0; s < 32; s += 16) {
        const uint32_t e = v >> s & 0xFFFFu;
        const bool is = which ? e == which : (e & 0x7F80u) == 0x7F80u && (e & 0x7Fu) != 0u;
        w |= is ? 0x3F80u << s : 0u;
    }
    return w;
}
template <int R>
__device__ __forceinline__ void add_odd(Rows<R>& w, const Keys& kv, const uint32_t (&seen)[R], uint32_t lane) {
#pragma unroll 1
    for (int k = 0; k < 3; ++k) {
        const uint32_t which = k == 0 ? 0x7F80u : k == 1 ? 0xFF80u : 0u;
        const float adds = k == 0 ? __builtin_inff() : k == 1 ? -__builtin_inff() : __builtin_nanf("");
        Keys ones;
#pragma unroll
        for (int i = 0; i < 8; ++i) ones.v[i] = uint2{ones_of_kind(kv.v[i].x, which), ones_of_kind(kv.v[i].y, which)};
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
                const f32x4 met = mfma16(v_operand(ones, i), sb, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (met[r] > 0.0f) w.o[rq][i][r] += adds;
            }
        }
    }
}

// What a workgroup works on. Nodes' keys follow the context's, in the same tiles.
struct Span {
    Nodes nodes;
    int32_t ctx, rows, all_tiles;  // of the sequence; rows = nodes x heads per KV head; tiles of TILE keys
};
template <int TILE>
__device__ __forceinline__ Span span_of(const TreeQueries& tq, int32_t b) {
    Span s;
    s.nodes = nodes_of(tq, b);
    s.ctx = context_of(tq, b);
    s.rows = s.nodes.count * tq.G;
    s.all_tiles = (s.ctx + s.nodes.count + TILE - 1) / TILE;
    return s;
}
// How many keys a tile has at most.
template <int TILE>
__device__ __forceinline__ uint32_t keys_from(const Span& s, int32_t t) {
    return (uint32_t)(s.ctx + s.nodes.count - t * TILE);
}
// One past the last tile that rows up to `last_row` look at (a chain's nodes end with their own).
template <int TILE>
__device__ __forceinline__ int32_t last_tile(const TreeQueries& tq, const Span& s, int32_t last_row) {
    if (tq.mask || last_row >= s.rows) return s.all_tiles;
    return (s.ctx + last_row / tq.G) / TILE + 1;
}

// The lane's rows row0 + 16 rq + l % 16: their queries, and their nodes (-1 past the last row).
template <int R>
__device__ __forceinline__ void load_rows(Rows<R>& w, int32_t (&node)[R], const TreeQueries& tq, const Span& s, int32_t h,
                                          int32_t row0, uint32_t lane, float c) {
#pragma unroll
    for (int rq = 0; rq < R; ++rq) {
        const int32_t r = row0 + 16 * rq + (int32_t)(lane & 15u);
        node[rq] = -1;
        w.q[rq][0] = w.q[rq][1] = U32x4{0u, 0u, 0u, 0u};
        if (r < s.rows) {
            node[rq] = r / tq.G;
            const uint16_t* q = tq.q + (int64_t)(s.nodes.first + node[rq]) * tq.q_rs +
                                (int64_t)(h * tq.G + r - node[rq] * tq.G) * tq.q_hs + 8 * (lane >> 4);
            w.q[rq][0] = load16(q);
            w.q[rq][1] = load16(q + 32);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w.o[rq][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        w.base[rq] = kNone;
        w.c[rq] = c;
        w.l[rq] = 0.0f;
    }
}

// Which of the 32 keys from key0 on each of the lane's rows sees.
template <int R>
__device__ __forceinline__ void seen_rows(uint32_t (&seen)[R], const int32_t (&node)[R], uint32_t exists,
                                          const TreeQueries& tq, const Span& s, int32_t key0) {
#pragma unroll
    for (int rq = 0; rq < R; ++rq) {
        uint32_t word[1];
        seen_keys<1>(word, tq, s.nodes, s.ctx, node[rq], key0);
        seen[rq] = exists & word[0];
    }
}

struct Factors {
    float c, capped;
};
template <bool CAP>
__device__ __forceinline__ Factors factors(const TreeQueries& tq) {
    return Factors{CAP ? 2.0f * kLog2E * tq.scale / tq.softcap : kLog2E * tq.scale, CAP ? tq.softcap * kLog2E : 0.0f};
}

// Where a row's results go: out and lse of row `at`, or, of one of several splits, its partial sums at
// row `at` of `o` [., 64] and `ml` [., 2].
struct Results {
    uint16_t* out;
    float* lse;
    float* o;
    float* ml;
    bool whole;
};
__device__ __forceinline__ void put_row4(const Results& t, int64_t at, int32_t d, float top, float l, f32x4 o) {
    const float base = top == -__builtin_inff() ? 0.0f : top;
    if (!t.whole) {
        *reinterpret_cast<f32x4*>(t.o + at * kHeadDim + d) = o;
        if (d == 0) {
            t.ml[at * 2] = top;
            t.ml[at * 2 + 1] = l;
        }
    } else {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint2 w;
        w.x = pack_bf16(o[0] * inv, o[1] * inv);
        w.y = pack_bf16(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2*>(t.out + at * kHeadDim + d) = w;
        if (d == 0) t.lse[at] = l == 0.0f ? -__builtin_inff() : (base + log2_hw(l)) * kLn2;
    }
}

// The rows that no sequence's nodes are: out 0 and lse -inf where `fill` asks for it (an out whose memory holds nothing
// yet), by workgroups of their own behind the attending ones, number `group` of `groups`. Those before the first
// sequence and behind the last are two runs of memory; sequences with rows past max_nodes (or with a range that does
// not lie in [0, T]) are looked for 64 at a time by every wave. No workgroup writes another's rows, so nothing is waited for.
__device__ __forceinline__ void fill_rows(const TreeQueries& tq, uint32_t fill, uint16_t* out, float* lse, uint32_t group,
                                          uint32_t groups) {
    const int64_t heads = tq.H * tq.G;
    // rows from .. to - 1, 16 bytes a thread, by `among` threads of which this is number `me`
    auto rows = [&](int64_t from, int64_t to, int64_t me, int64_t among) {
        if (fill & NRC_ATTENTION_FILL_OUT)
            for (int64_t i = from * heads * 8 + me; i < to * heads * 8; i += among) store16(out + 8 * i, U32x4{0u, 0u, 0u, 0u});
        if (fill & NRC_ATTENTION_FILL_LSE)
            for (int64_t i = from * heads + me; i < to * heads; i += among) lse[i] = -__builtin_inff();
    };
    const int64_t me = (int64_t)group * blockDim.x + threadIdx.x, among = (int64_t)groups * blockDim.x;
    const int32_t begin = tq.B > 0 ? tq.q_starts[0] : tq.T, end = tq.B > 0 ? tq.q_starts[tq.B] : tq.T;
    rows(0, begin > tq.T ? tq.T : begin, me, among);
    rows(end < 0 ? 0 : end, tq.T, me, among);
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    for (int64_t b0 = me - lane; b0 < tq.B; b0 += among) {
        int32_t from = 0, to = 0;
        if (b0 + lane < tq.B) {
            const int32_t b = (int32_t)b0 + lane, lo = tq.q_starts[b], hi = tq.q_starts[b + 1];
            from = (lo < 0 ? 0 : lo) + nodes_of(tq, b).count;
            to = hi > tq.T ? tq.T : hi;
        }
        for (uint64_t left = __ballot(from < to); left != 0; left &= left - 1) {
            const int l = __builtin_ctzll(left);
            rows(__builtin_amdgcn_readlane(from, l), __builtin_amdgcn_readlane(to, l), lane, 64);
        }
    }
}

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// What a wave of the many-rows kernel carries for R query tiles of 32 rows.
// Scores come as S^T = K Q^T by v_mfma_f32_32x32x16_bf16: lane l holds, for
// row l % 32, the keys 8 (i / 4) + 4 (l / 32) + i % 4 of 32 at i = 0 .. 15; slot 8
// (l / 32) + j of step ks of the second product stands for the key at i = 8 ks + j.
template <int R>
struct Rows32 {
    U32x4 q[R][4];   // row l % 32, d = 16 i + 8 (l / 32) ...
    f32x16 o[R][2];  // O^T: row l % 32, d = 32 c + 8 (i / 4) + 4 (l / 32) + i % 4 at [c][i]
    float base[R], c[R], l[R];  // as Rows'

};
struct Keys32 {
    U32x4 k[4];     // key l % 32, d as q's
    U32x4 v[2][2];  // [c][ks]: d = 32 c + l % 32, the keys of slots 8 (l / 32) .. + 7 of step ks
};

template <int R, bool CAP>
__device__ __forceinline__ void raise32(Rows32<R>& w, int rt, const f32x16& s, float c, float capped) {
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, s[i]);
    top = __builtin_fmaxf(top, lane_xor<32>(top));
    const float shrink = rebase<CAP>(top, w.base[rt], w.c[rt], c, capped);
    w.l[rt] *= shrink;
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) w.o[rt][d][i] *= shrink;
}

// The weights of 16 scores, as the second product's operands (rounded as open_weights says), and their sum.
// seen: bit i of a masked tile's scores.
template <bool CAP, bool MASKED>
__device__ __forceinline__ float weights32(const f32x16& s, float base, float c, float capped, uint32_t seen,
                                           U32x4 (&pb)[2]) {
    const float from = CAP ? capped - base : -base;
    float p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        p[i] = exp2_hw(CAP ? __builtin_fmaf(rcp_hw(exp2_hw(s[i] * c) + 1.0f), -2.0f * capped, from)
                           : __builtin_fmaf(s[i], c, from));
        // (bit i over the whole word, and its float)
        if (MASKED) p[i] = __uint_as_float(__float_as_uint(p[i]) & (uint32_t)__builtin_amdgcn_sbfe((int)seen, i, 1));
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
        pb[ks] = U32x4{pack_bf16_pair_hw(p[8 * ks], p[8 * ks + 1]), pack_bf16_pair_hw(p[8 * ks + 2], p[8 * ks + 3]),
                       pack_bf16_pair_hw(p[8 * ks + 4], p[8 * ks + 5]), pack_bf16_pair_hw(p[8 * ks + 6], p[8 * ks + 7])};
    float sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = (p[4 * i] + p[4 * i + 1]) + (p[4 * i + 2] + p[4 * i + 3]);
    return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

template <int R>
__device__ __forceinline__ void scores32(f32x16& s, const Rows32<R>& w, int rt, const Keys32& kv) {
    s = f32x16{0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) s = mfma32(kv.k[i], w.q[rt][i], s);
}
// Weights of row tile rt's scores, its sum, and V by them.
template <int R, bool CAP, bool MASKED>
__device__ __forceinline__ void add32(Rows32<R>& w, int rt, f32x16& s, const Keys32& kv, const Factors& f,
                                      uint32_t seen) {
    U32x4 pb[2];
    float sum = weights32<CAP, MASKED>(s, w.base[rt], CAP ? f.c : w.c[rt], f.capped, seen, pb);
    if (__any(!(sum <= kMost))) {
        if constexpr (MASKED) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (!(seen >> i & 1u)) s[i] = -__builtin_inff();
        }
        raise32<R, CAP>(w, rt, s, f.c, f.capped);
        sum = weights32<CAP, MASKED>(s, w.base[rt], CAP ? f.c : w.c[rt], f.capped, seen, pb);
    }
    w.l[rt] += sum;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) w.o[rt][c] = mfma32(kv.v[c][ks], pb[ks], w.o[rt][c]);
}

// How a batch whose workgroups fit the chip at once is split: into shares of
// at most `tiles` tiles of KEYS keys, the least for which all of them are at most
// `most`, so that ragged sequences end together (no share is smaller than `least`). Worked out by every wave
// from the lengths (B <= 512).
struct Shares {
    int32_t tiles, groups;          // of a share; of all sequences and heads
    int32_t b, h, split, splits;    // of group g (b < 0: there is none)
    int32_t first;                  // of the sequence: its first group
};
template <int KEYS>
__device__ __forceinline__ Shares shares_of(const TreeQueries& tq, int32_t most, int32_t least, int32_t g, uint32_t lane) {
    constexpr int kSets = 8;
    int32_t tiles[kSets];
    int32_t sum = 0, longest = 0;
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
        tiles[j] = 0;
        const int32_t b = 64 * j + (int32_t)lane;
        if (64 * j < tq.B && b < tq.B) {
            const Span s = span_of<KEYS>(tq, b);
            tiles[j] = s.rows > 0 ? s.all_tiles : 0;
        }
        sum += tiles[j];
        longest = longest > tiles[j] ? longest : tiles[j];
    }
    sum = (int32_t)wave_total((uint32_t)sum);
    longest = (int32_t)wave_most((uint32_t)longest);
    auto count = [&](int32_t c) {
        int32_t n = 0;
#pragma unroll
        for (int j = 0; j < kSets; ++j)
            if (64 * j < tq.B) n += (tiles[j] + c - 1) / c;
        return (int32_t)wave_total((uint32_t)n) * tq.H;
    };
    int32_t lo = (int32_t)(((int64_t)sum * tq.H + most - 1) / most), hi = longest;
    if (lo < least) lo = least;  // (no share is smaller)
    while (lo < hi) {
        const int32_t mid = (lo + hi) / 2;
        if (count(mid) <= most)
            hi = mid;
        else
            lo = mid + 1;
    }
    Shares r{lo, 0, -1, 0, 0, 1, 0};
    int32_t before = 0;  // groups of the sequences before
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
        if (64 * j >= tq.B) break;
        const int32_t n = (tiles[j] + lo - 1) / lo * tq.H;
        const int32_t upto = before + (int32_t)wave_inclusive((uint32_t)n);
        const uint64_t past = __ballot(upto > g);
        if (r.b < 0 && past != 0) {
            const int32_t l = __builtin_ctzll(past);
            r.b = 64 * j + l;
            const int32_t mine = __builtin_amdgcn_readlane(n, l);
            r.first = __builtin_amdgcn_readlane(upto, l) - mine;
            r.splits = mine / tq.H;
            r.h = (g - r.first) / r.splits;
            r.split = (g - r.first) - r.h * r.splits;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    r.groups = before;
    return r;
}

}  // namespace
}  // namespace nrc
