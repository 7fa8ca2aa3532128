// The attention weight that cached cells receive: out_j = decay w_j + sum over
// the KV head's query rows i that see key j of e^(s_ij - lse_i), lse from the
// attention's forward pass. Cells at and past the sequence's end become 0.
//
// Keys stay, queries pass: a wave keeps the K of KT tiles of 32 keys as A
// operands (S^T = K Q^T, v_mfma_f32_32x32x16_bf16), a workgroup's waves share the
// query rows, staged in LDS kStage at a time in two buffers (global_load_lds).
// Each lane adds its rows' exponentials to the keys it holds, and the 32 rows'
// lanes are summed at the end. A key belongs to one wave, so the sums have one
// order and no atomics. Bound by the vector unit, busy 87% of the time: an FMA, an
// exponential and an FMA a score (16 cycles a wave's 64; 48 instructions to 32 keys by 32 rows) and 40 more around
// them (the stage's addresses, the rows' factors, the loop). 16 sequences of up to 16384 keys, 512 rows a head: 69
// GFLOP in 138 us.
// e^(s - lse) = 2^(c s + m) with c = scale log2 e and m = -c lse / scale rounded
// to FP32: what the rounding lost, 2^(lost), is the factor of the last FMA. c's own rounding then meets s - lse alone, which is small near the
// largest weights, so the weights keep FP32's relative accuracy. (Past 2^30 the
// lost part alone would overflow, while scores that differ at all are 2^7 apart and
// more: c's power of two takes its place, exact where a score equals lse.)
// Few keys (less than two workgroups a CU): KT 1, for twice the workgroups.
#include <type_traits>

#include "cache_ops.h"
#include "paged.h"

namespace nrc {
namespace {

// tanh by Lambert's continued fraction, its x taken out so that small arguments
// keep their relative accuracy: cut after 5 levels, x - x^3 (315 + 14 x^2) / (945
// + 420 x^2 + 15 x^4), off by 1e-8 at |x| = 0.7; after 7 levels off by 1e-7 at 2;
// beyond, 1 - 2 / (e^2x + 1).
constexpr float kNear = 0.7f;
__device__ __forceinline__ float tanh_near(float x) {
    const float x2 = x * x;
    const float num = __builtin_fmaf(14.0f, x2, 315.0f);
    const float den = __builtin_fmaf(__builtin_fmaf(15.0f, x2, 420.0f), x2, 945.0f);
    return __builtin_fmaf(-(x * x2), num * rcp_hw(den), x);
}
__device__ __forceinline__ float tanh_of(float x) {
    const float x2 = x * x;
    const float num = __builtin_fmaf(__builtin_fmaf(27.0f, x2, 2772.0f), x2, 45045.0f);
    const float den = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(28.0f, x2, 3150.0f), x2, 62370.0f), x2, 135135.0f);
    const float near = __builtin_fmaf(-(x * x2), num * rcp_hw(den), x);
    const float far = __builtin_fmaf(rcp_hw(exp2_hw(x * (2.0f * kLog2E)) + 1.0f), -2.0f, 1.0f);
    return __builtin_fabsf(x) < 2.0f ? near : far;
}

// Grid (blocks of keys, H, B), 4 waves of 32 KT keys each.
constexpr int kStage = 64, kRuns = kStage / 32;  // query rows; runs of 8 of them a wave brings in
template <int KT, bool CAP>
__global__ __launch_bounds__(256, CAP ? (KT == 1 ? 3 : 2) : (KT == 1 ? 4 : 3)) void attention_mass_kernel(PagedCache kv, TreeQueries tq,
                                                             const float* __restrict__ lse, const float* weights,
                                                             int64_t w_bs, int64_t w_hs, float decay, float* out,
                                                             int64_t out_bs, int64_t out_hs, int64_t width) {
    // rows of 128 bytes, 16-byte chunk c at c ^ (row & 7): 8 lanes reading one chunk of 8 rows meet all banks
    __shared__ __attribute__((aligned(16))) uint8_t stage[2][kStage * 128];
    __shared__ __attribute__((aligned(16))) float stage_lse[2][kStage];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t hl = lane >> 5, n32 = lane & 31u;
    const int32_t h = blockIdx.y, b = blockIdx.z;
    const int32_t block0 = (int32_t)blockIdx.x * 128 * KT, key0 = block0 + (int32_t)wave * 32 * KT;
    const uint16_t* head = kv.cache + (int64_t)h * kv.head_stride;
    const int32_t* table = kv.tables + (int64_t)b * kv.table_stride;
    // On the way before the lengths are known: the keys' table entries, and the earlier weights (of few query rows a
    // workgroup's time is its chain of loads).
    const int64_t at_w = b * w_bs + h * w_hs, at_o = b * out_bs + h * out_hs;
    const int32_t own = (int32_t)(8 * (lane >> 3 & 3u) + 4 * hl + (lane >> 1 & 3u));  // of 32 keys, the lane's in the end
    uint32_t page[KT];
    float earlier[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
        page[kt] = page_of(kv, table, (uint32_t)(key0 + 32 * kt) + n32);
        const int64_t key = key0 + 32 * kt + own;
        earlier[kt] = weights && key < width ? weights[at_w + key] : 0.0f;
    }
    const Nodes nodes = nodes_of(tq, b);
    const int32_t ctx = context_of(tq, b);
    const int32_t rows = nodes.count * tq.G, total = ctx + nodes.count, heads = tq.H * tq.G;
    const bool any = block0 < total && rows > 0;  // (the same in the workgroup)

    // Rows of the stage that the lane brings in: of Q, in run i of the wave (8 rows), row lane / 8 and the chunk that
    // belongs in place lane % 8; wave 0 also row `lane`'s lse. They move on by a stage at a time, addresses by fixed
    // steps: a division, or a product of strides, a stage would cost as much as its exponentials.
    const int32_t step_node = kStage / tq.G, step_in = kStage - step_node * tq.G;
    const int64_t q_step = step_node * tq.q_rs + step_in * tq.q_hs, q_wrap = tq.q_rs - tq.G * tq.q_hs;
    const int32_t l_step = step_node * heads + step_in;
    // r / G for r < 64: 2^32 / G rounded up, times r (G = 1: r itself)
    const uint32_t g_inv = tq.G > 1 ? 0xFFFFFFFFu / (uint32_t)tq.G + 1u : 0u;
    auto per_group = [&](int32_t r) { return g_inv ? (int32_t)__umulhi((uint32_t)r, g_inv) : r; };
    const uint32_t row8 = lane >> 3, c8 = lane & 7u, lds0 = lds_address(stage), lds_l = lds_address(stage_lse);
    const uint16_t* q0 = tq.q + nodes.first * tq.q_rs + (int64_t)h * tq.G * tq.q_hs + 8 * (c8 ^ row8);
    const float* l0 = lse + (int64_t)nodes.first * heads + h * tq.G;
    const uint16_t* q_at[kRuns];
    int32_t q_row[kRuns], q_in[kRuns];
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
        q_row[i] = (int32_t)(8 * (kRuns * wave + i) + row8);
        const int32_t node = per_group(q_row[i]);
        q_in[i] = q_row[i] - node * tq.G;
        q_at[i] = q0 + node * tq.q_rs + q_in[i] * tq.q_hs;
    }
    int32_t l_row = (int32_t)lane, l_in, l_at;
    {
        const int32_t node = per_group(l_row);
        l_in = l_row - node * tq.G;
        l_at = node * heads + l_in;
    }
    auto bring = [&](int buf) {
        // (past the end the first row, which is masked)
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            to_lds(q_row[i] < rows ? q_at[i] : q0, lds0 + buf * (kStage * 128) + (kRuns * wave + i) * 1024);
            q_row[i] += kStage;
            q_in[i] += step_in;
            q_at[i] += q_step;
            if (q_in[i] >= tq.G) {
                q_in[i] -= tq.G;
                q_at[i] += q_wrap;
            }
        }
        if (wave == 0) {
            to_lds4(l_row < rows ? l0 + l_at : l0, lds_l + buf * (kStage * 4));
            l_row += kStage;
            l_in += step_in;
            l_at += l_step;
            if (l_in >= tq.G) {
                l_in -= tq.G;
                l_at += heads - tq.G;
            }
        }
    };
    if (any) {
        bring(0);
    }

    f32x16 acc[KT];
    U32x4 k[KT][4];
    uint32_t exists[KT];
    bool plain = key0 + 32 * KT <= ctx;  // every row sees every key of the wave
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
        const int32_t key = key0 + 32 * kt + (int32_t)n32;
        int64_t off = -1;
        if (key < total) off = key_offset(kv, (uint32_t)key, page[kt]);
        exists[kt] = (uint32_t)__ballot(off >= 0);
        plain &= exists[kt] == 0xFFFFFFFFu;
        // (a key that is not there is read from the cache's first cell, and masked)
        const uint16_t* at = head + (off >= 0 ? off : 0) + 8 * hl;
#pragma unroll
        for (int i = 0; i < 4; ++i) k[kt][i] = load16(at + 16 * i);
        acc[kt] = f32x16{0.f};
    }

    const float inv_cap = CAP ? tq.scale / tq.softcap : 0.0f, inv_scale = 1.0f / tq.scale;
    const float c = tq.scale * kLog2E, c_power = __uint_as_float(__float_as_uint(c) & 0x7F800000u);
    if (any) {
        // Of 32 rows at row0: the factors of their weights, and Q as B operands.
        struct Part {
            float c, m, f;
            int32_t row;
            bool masked, live;
        };
        U32x4 q[4];
        const uint32_t q_place = n32 * 128 + ((hl ^ (n32 & 7u)) << 4);
        auto begin = [&](int32_t row0) {
            const int part = row0 / 32 & (kStage / 32 - 1), buf = row0 / kStage & 1;
            if (part == 0) {
                landed();
                if (row0 + kStage < rows) bring(buf ^ 1);
            }
            const float l = stage_lse[buf][32 * part + n32];
            Part x;
            x.row = row0 + (int32_t)n32;
            x.live = x.row < rows && l != -__builtin_inff();  // rows past the end, and rows that saw nothing, add 0
            x.masked = !plain || __any(!x.live);
            const float at = -l * inv_scale;
            x.c = c;
            x.m = CAP ? -l : at * c;
            x.f = 1.0f;
            if constexpr (!CAP) {
                if (__builtin_fabsf(x.m) > 0x1p30f) {
                    x.c = c_power;
                    x.m = at * c_power;
                } else {
                    x.f = exp2_hw(__builtin_fmaf(at, c, -x.m));
                }
            }
            const uint8_t* from = &stage[buf][part * 4096];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = load16(from + (q_place ^ j * 32));
            return x;
        };
        auto scores = [&](f32x16& s, int kt) {
            s = f32x16{0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) s = mfma32(k[kt][j], q[j], s);
        };
        auto add = [&](const f32x16& s, int kt, const Part& x) {
            float p[16];
            if constexpr (CAP) {
                float t[16], most = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    t[j] = s[j] * inv_cap;
                    most = __builtin_fmaxf(most, __builtin_fabsf(t[j]));
                }
                // (a NaN beside near ones goes through tanh_near as NaN)
                if (__any(most >= kNear)) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) t[j] = tanh_of(t[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) t[j] = tanh_near(t[j]);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) p[j] = exp2_hw(__builtin_fmaf(tq.softcap, t[j], x.m) * kLog2E);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) p[j] = exp2_hw(__builtin_fmaf(s[j], x.c, x.m));
            }
            if (x.masked) {
                uint32_t seen = 0u;
                if (x.live) {
                    uint32_t word[1];
                    seen_keys<1>(word, tq, nodes, ctx, x.row / tq.G, key0 + 32 * kt);
                    seen = exists[kt] & word[0];
                }
                seen = bits_of_scores(seen, hl);
#pragma unroll
                for (int j = 0; j < 16; ++j) p[j] = seen >> j & 1u ? p[j] : 0.0f;
            }
            const float f = x.live ? x.f : 0.0f;  // (lse -inf makes f NaN)
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[kt][j] = __builtin_fmaf(p[j], f, acc[kt][j]);
        };
        // The matrix cores work out one tile's scores while the vector unit takes the other's exponentials.
        f32x16 s0, s1;
        Part x = begin(0);
        scores(s0, 0);
#pragma unroll 1
        for (int32_t row0 = 0; row0 < rows; row0 += 32) {
            const bool more = row0 + 32 < rows;
            if constexpr (KT == 2) {
                scores(s1, 1);
                add(s0, 0, x);
                Part y = x;
                if (more) {
                    y = begin(row0 + 32);
                    scores(s0, 0);
                }
                add(s1, 1, x);
                x = y;
            } else {
                add(s0, 0, x);
                if (more) {
                    x = begin(row0 + 32);
                    scores(s0, 0);
                }
            }
        }
    }
    // The sums over the 32 lanes of a half: each exchange halves the keys a lane
    // holds; bits 4 .. 1 of the lane name the one it ends with.
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = acc[kt][i];
        auto halve = [&](auto mask, int n) {
            constexpr int M = decltype(mask)::value;
            const bool upper = lane & M;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= n) break;
                const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
                v[i] = keep + lane_xor<M>(give);
            }
        };
        halve(std::integral_constant<int, 16>{}, 8);
        halve(std::integral_constant<int, 8>{}, 4);
        halve(std::integral_constant<int, 4>{}, 2);
        halve(std::integral_constant<int, 2>{}, 1);
        float mass = v[0] + lane_xor<1>(v[0]);
        // (halving: bit 4 chose i's bit 3, bit 3 its bit 2, bit 2 its bit 1, bit 1 its bit 0)
        const int64_t key = key0 + 32 * kt + own;
        if ((lane & 1u) == 0u && key < width) {
            if (key >= total)
                mass = 0.0f;
            else if (weights)
                mass = __builtin_fmaf(earlier[kt], decay, mass);
            out[at_o + key] = mass;
        }
    }
}

template <int KT>
void launch_kt(const AttentionMassArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)((a.width + 128 * KT - 1) / (128 * KT)), (uint32_t)a.tq.H, (uint32_t)a.tq.B);
    auto kernel = a.tq.softcap > 0.0f ? attention_mass_kernel<KT, true> : attention_mass_kernel<KT, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a.kv, a.tq, a.lse, a.weights, a.w_bs, a.w_hs, a.decay,
                       a.out, a.out_bs, a.out_hs, a.width);
}

}  // namespace

int launch_attention_mass(const AttentionMassArgs& a, hipStream_t stream) {
    const int64_t blocks = (a.width + 255) / 256 * a.tq.H * a.tq.B;
    if (blocks < 2 * (int64_t)a.num_cus)
        launch_kt<1>(a, stream);
    else
        launch_kt<2>(a, stream);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
