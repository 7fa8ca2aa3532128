// The attention weight that cached cells receive: out_j = decay w_j + sum over
// the KV head's query rows i that see key j of e^(s_ij - lse_i), lse from the
// attention's forward pass. Cells at and past the sequence's end become 0.
//
// Keys stay, queries pass: a wave keeps the K of KT tiles of 16 keys as A
// operands (S^T = K Q^T, as in the attention kernel) and goes over the query rows
// 16 at a time; each lane adds its scores' exponentials to the keys it holds.
// A key belongs to one wave, so the sums have one order and no atomics.
// The difference s - lse is one FMA (scale s - lse) ahead of the exponential's
// own factor log2 e: near the largest weights it is small, so the weight's
// relative error stays near FP32's.
#include "cache_ops.h"
#include "paged.h"

namespace nrc {
namespace {

// tanh: x - x^3 (45045 + 2772 x^2 + 27 x^4) / (135135 + 62370 x^2 + 3150 x^4
// + 28 x^6) for |x| < 2 (Lambert's continued fraction cut after 7 levels, its
// x taken out so that small arguments keep their relative accuracy; off by
// 1e-7 at 2), 1 - 2 / (e^2x + 1) beyond.
__device__ __forceinline__ float tanh_of(float x) {
    const float x2 = x * x;
    const float num = __builtin_fmaf(__builtin_fmaf(27.0f, x2, 2772.0f), x2, 45045.0f);
    const float den = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(28.0f, x2, 3150.0f), x2, 62370.0f), x2, 135135.0f);
    const float near = __builtin_fmaf(-(x * x2), num * rcp_hw(den), x);
    const float far = __builtin_fmaf(rcp_hw(exp2_hw(x * (2.0f * kLog2E)) + 1.0f), -2.0f, 1.0f);
    return __builtin_fabsf(x) < 2.0f ? near : far;
}

// Bits 0 .. 15: does node i (row `row`) see keys key0 .. key0 + 15 of a
// sequence with ctx keys of context and n nodes.
__device__ __forceinline__ uint32_t seen16(const TreeQueries& t, int32_t row, int32_t i, int32_t n, int32_t ctx,
                                           int32_t key0) {
    const int32_t j0 = key0 - ctx;
    if (j0 <= -16) return 0xFFFFu;
    if (j0 >= n) return 0u;
    if (j0 < 0) return ((1u << -j0) - 1u) | (seen_word(t, row, i, n, 0) << -j0 & 0xFFFFu);
    const int32_t w = j0 >> 5, s = j0 & 31;
    uint32_t bits = seen_word(t, row, i, n, w) >> s;
    if (s > 16) bits |= seen_word(t, row, i, n, w + 1) << (32 - s);
    return bits & 0xFFFFu;
}

// Grid (blocks of keys, H, B), 4 waves of 16 KT keys each.
template <int KT, bool CAP>
__global__ __launch_bounds__(256) void attention_mass_kernel(PagedCache kv, TreeQueries tq,
                                                             const float* __restrict__ lse, const float* weights,
                                                             int64_t w_bs, int64_t w_hs, float decay, float* out,
                                                             int64_t out_bs, int64_t out_hs, int64_t width) {
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t g = lane >> 4, n16 = lane & 15u;
    const int32_t h = blockIdx.y, b = blockIdx.z;
    const Nodes nodes = nodes_of(tq, b);
    const int32_t ctx = context_of(tq, b);
    const int32_t rows = nodes.count * tq.G, total = ctx + nodes.count, heads = tq.H * tq.G;
    const int32_t key0 = ((int32_t)blockIdx.x * 4 + (int32_t)wave) * 16 * KT;
    const uint16_t* head = kv.cache + (int64_t)h * kv.head_stride;
    const int32_t* table = kv.tables + (int64_t)b * kv.table_stride;

    float acc[KT][4];
    U32x4 k[KT][2];
    uint32_t exists[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
        const int32_t key = key0 + 16 * kt + (int32_t)n16;
        int64_t off = -1;
        if (key < total) off = key_offset(kv, table, (uint32_t)key);
        exists[kt] = (uint32_t)__ballot(off >= 0) & 0xFFFFu;
        k[kt][0] = k[kt][1] = U32x4{0u, 0u, 0u, 0u};
        if (off >= 0) {
            k[kt][0] = load16(head + off + 8 * g);
            k[kt][1] = load16(head + off + 32 + 8 * g);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[kt][r] = 0.0f;
    }
    bool plain = key0 + 16 * KT <= ctx;  // every row sees every key of the wave
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) plain &= exists[kt] == 0xFFFFu;

    if (key0 < total) {
        const float inv_cap = CAP ? tq.scale / tq.softcap : 0.0f;
        for (int32_t row0 = 0; row0 < rows; row0 += 16) {
            const int32_t r0 = row0 + (int32_t)n16;
            U32x4 q[2] = {U32x4{0u, 0u, 0u, 0u}, U32x4{0u, 0u, 0u, 0u}};
            float minus = -__builtin_inff();  // - lse; rows past the end, and rows that saw nothing, add 0
            int32_t node = 0;
            if (r0 < rows) {
                node = r0 / tq.G;
                const int64_t row = nodes.first + node;
                const int32_t hq = h * tq.G + r0 - node * tq.G;
                const uint16_t* p = tq.q + row * tq.q_rs + (int64_t)hq * tq.q_hs + 8 * g;
                q[0] = load16(p);
                q[1] = load16(p + 32);
                const float l = lse[row * heads + hq];
                if (l != -__builtin_inff()) minus = -l;
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                f32x4 s = mfma16(k[kt][0], q[0], f32x4{0.f, 0.f, 0.f, 0.f});
                s = mfma16(k[kt][1], q[1], s);
                uint32_t seen = 0xFFFFu;
                if (!plain)
                    seen = exists[kt] & seen16(tq, nodes.first + node, node, nodes.count, ctx, key0 + 16 * kt);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float d = CAP ? __builtin_fmaf(tq.softcap, tanh_of(s[r] * inv_cap), minus)
                                  : __builtin_fmaf(s[r], tq.scale, minus);
                    if (!plain && !(seen >> (4 * g + r) & 1u)) d = -__builtin_inff();
                    acc[kt][r] += exp2_hw(d * kLog2E);
                }
            }
        }
    }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v = acc[kt][r];
            v = v + lane_xor<1>(v);
            v = v + lane_xor<2>(v);
            v = v + lane_xor<4>(v);
            v = v + lane_xor<8>(v);
            const int64_t key = key0 + 16 * kt + 4 * (int32_t)g + r;
            if (n16 == (uint32_t)(4 * (kt % 4) + r) && key < width) {
                if (key >= total)
                    v = 0.0f;
                else if (weights)
                    v = __builtin_fmaf(weights[b * w_bs + h * w_hs + key], decay, v);
                out[b * out_bs + h * out_hs + key] = v;
            }
        }
    }
}

template <int KT>
void launch_kt(const AttentionMassArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)((a.width + 64 * KT - 1) / (64 * KT)), (uint32_t)a.tq.H, (uint32_t)a.tq.B);
    auto kernel = a.tq.softcap > 0.0f ? attention_mass_kernel<KT, true> : attention_mass_kernel<KT, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a.kv, a.tq, a.lse, a.weights, a.w_bs, a.w_hs, a.decay,
                       a.out, a.out_bs, a.out_hs, a.width);
}

}  // namespace

int launch_attention_mass(const AttentionMassArgs& a, hipStream_t stream) {
    launch_kt<4>(a, stream);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
